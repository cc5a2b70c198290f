// orth_small.cuh -- Newton-Schulz steps of small matrices, one block per matrix, and the TTT-Linear
// step whose inner update is orthogonalised (its gradient, its update, the general output pass).
//
// A matrix of at most 64 rows stays in shared memory through all steps, so nothing but the input and
// the result touches HBM.  Each operand lies there as 128 rows, 64 of hi and 64 of lo (fp16, as in
// orth.cuh), and one tcgen05 product of the stacked rows, [hi; lo] [hi | lo], gives hi hi, hi lo, lo hi and
// lo lo at once as quarters of a 128 x 128 accumulator: four MMAs of K = 16 for a 64 x 64 x 64 product,
// 268 cycles.  lo hi and lo lo sit in the lanes that the other warps can read, so each side of the block sends
// the other side's columns through shared memory; a thread finishes 16 columns of a row.
//
// X <- a X + P X with P = b A + c A^2: a X is added in fp32, so that the accumulator cuts and P's storage rounds only
// what the step adds, little in the first steps, whose errors are enlarged most.  With a in P's diagonal, and lo lo
// left out, fp32 results were 1.3 to 2.5 times as far off as the same steps in plain fp32: 64 x 64 1.9e-6 of the norm
// against 1.2e-6, 64 x 256 3.7e-6 against 1.5e-6; now 1.0e-6 and 2.4e-6 (two accumulators for X X^T: 2.2e-6).
//
// The bound is latency: a step is three such products, each waiting for the one before (accumulator
// out of tensor memory, exchange, rounding to hi + lo, operand written, MMAs; about 1400 cycles).  Several
// blocks share an SM and fill one another's gaps.  Compiled for two blocks an SM nothing spills (32 units of
// the TTT-Linear step, when measured: 27 us against 30 with three, 22 since); with more matrices than two blocks
// an SM hold, three make one wave of up to 444 (384 units: 41 us against 51).
#pragma once
#include "common.cuh"
#include "orth.cuh"

namespace orth {

constexpr int SM_M = 64;                 // rows of a small matrix
constexpr int SM_N = 256;                // its longer side at most
constexpr int SM_TPB = 256;              // 8 warps, two for each quarter of the accumulator's lanes
constexpr int SM_OP = 2 * SM_M * 128;    // an operand of 64 columns: 64 rows of hi, 64 of lo, 128-byte swizzle
constexpr int SM_EX = SM_M * SM_M * 4;   // the exchange
struct SmallBars {
    uint64_t done;
    uint32_t tmem_base;
    double sums[SM_TPB / 32];
};
__host__ __device__ constexpr int sm_strips(int N) { return (N + 63) / 64; }
// X (a strip per 64 columns), A and P, the exchange
constexpr int small_smem_bytes(int N) { return (sm_strips(N) + 1) * SM_OP + SM_EX + (int)sizeof(SmallBars) + 1024; }
constexpr uint32_t SM_IDESC_K = tc::idesc_f16(128, 128, 0, 0), SM_IDESC_MN = tc::idesc_f16(128, 128, 0, 1);

// 8 adjacent values into an operand at (row, col), col a multiple of 8
__device__ __forceinline__ void put_op8(uint8_t* op, int row, int col, const float* v) {
    uint2 h0, l0, h1, l1;
    const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
    split4(a, h0, l0);
    split4(b, h1, l1);
    uint8_t* at = op + swz<3>((uint32_t)row * 128 + (uint32_t)col * 2);
    *reinterpret_cast<uint4*>(at) = make_uint4(h0.x, h0.y, h1.x, h1.y);
    *reinterpret_cast<uint4*>(at + SM_M * 128) = make_uint4(l0.x, l0.y, l1.x, l1.y);
}

// what an operand holds there, hi + lo
__device__ __forceinline__ void get_op8(const uint8_t* op, int row, int col, float* v) {
    const uint8_t* at = op + swz<3>((uint32_t)row * 128 + (uint32_t)col * 2);
    const uint4 h = *reinterpret_cast<const uint4*>(at), l = *reinterpret_cast<const uint4*>(at + SM_M * 128);
    const uint32_t hi[4] = {h.x, h.y, h.z, h.w}, lo[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&hi[e])), b = __half22float2(*reinterpret_cast<const __half2*>(&lo[e]));
        v[2 * e] = a.x + b.x;
        v[2 * e + 1] = a.y + b.y;
    }
}

// What a block works with
struct Small {
    uint8_t *X, *A;    // strips of X; A, then P
    float* ex;
    SmallBars* bars;
    uint32_t tmem;
    int products;      // products waited for so far (the barrier's phase)

    __device__ __forceinline__ void begin(uint8_t* raw, int strips) {
        X = smem_align<1024>(raw);
        A = X + strips * SM_OP;
        ex = reinterpret_cast<float*>(A + SM_OP);
        bars = reinterpret_cast<SmallBars*>(A + SM_OP + SM_EX);
        products = 0;
        if (threadIdx.x == 0) {
            mbar_init(&bars->done, 1);
            mbar_fence_init();
        }
        if (threadIdx.x < 32) tc::alloc(&bars->tmem_base, 128);
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
        tmem = bars->tmem_base;
    }
    __device__ __forceinline__ void end() {
        tc::fence_before();
        __syncthreads();
        if (threadIdx.x < 32) tc::dealloc(tmem, 128);
    }
    // The operands that the block has written are seen by the tensor cores, and the accumulator has been read
    __device__ __forceinline__ void written() {
        fence_proxy_async_smem();
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
    }
    // The row and the first of the 16 columns that a thread finishes: warps 0, 1, 4, 5 read the lanes of hi hi
    // and hi lo and finish columns 0 .. 31, the others read those of lo hi and lo lo and finish columns 32 .. 63.
    static __device__ __forceinline__ int row() { return (threadIdx.x >> 5 & 1) * 32 + (threadIdx.x & 31); }
    static __device__ __forceinline__ int col() { return (threadIdx.x >> 6 & 1) * 32 + (threadIdx.x >> 7) * 16; }
    // v: the thread's values of hi hi + hi lo + lo hi + lo lo
    __device__ __forceinline__ void take(float (&v)[16]) {
        mbar_wait<false>(&bars->done, products++ & 1, TTT_DEVERR_TIMEOUT_TMA);
        tc::fence_after();
        const int warp = threadIdx.x >> 5, side = warp >> 1 & 1, c0 = (warp >> 2) * 16;
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
        // this side's columns and the other side's: side 0 keeps the first half and sends the second
        const uint32_t mine = at + 32 * side, theirs = at + 32 - 32 * side;
        float s[16], h[16], l[16];
        tc::ld16(mine, v);
        tc::ld16(theirs, s);
        tc::ld16(mine + 64, h);
        tc::ld16(theirs + 64, l);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            v[c] += h[c];
            s[c] += l[c];
        }
        float* out = ex + (side * 32 + c0) * SM_M + row();  // [column][row]
        const float* in = ex + ((1 - side) * 32 + c0) * SM_M + row();
#pragma unroll
        for (int c = 0; c < 16; ++c) out[c * SM_M] = s[c];
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] += in[c * SM_M];
    }

    // All steps on X (written, not yet synchronised); the last product goes to last(row, column, v): 16 adjacent
    // values of X, times SX SP.
    template <typename Last>
    __device__ __forceinline__ void steps(int strips, int count, float ca, float cb, float cc, Last last) {
        const int row = this->row(), col = this->col();
        const uint64_t xk = tc::smem_desc(smem_u32(X), 16, 1024, 2), xn = tc::smem_desc(smem_u32(X), SM_M * 128, 1024, 2);
        const uint64_t ak = tc::smem_desc(smem_u32(A), 16, 1024, 2);
        const float pa = SP * ca, pb = SP / SX * cb, pc = SP / (SX * SX) * cc;  // P = SP (b A + c A^2)
        for (int k = 0; k < count; ++k) {
            float v[16], a[16];
            written();
            if (threadIdx.x == 0) {
                for (int s = 0; s < strips; ++s)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t d = xk + (uint64_t)(s * (SM_OP >> 4) + 2 * ks);
                        tc::mma_bf16(tmem, d, d, SM_IDESC_K, s > 0 || ks > 0);
                    }
                tc::commit(&bars->done);
            }
            take(a);
#pragma unroll
            for (int c = 0; c < 16; ++c) a[c] *= 1.f / SX;  // A as it is stored
#pragma unroll
            for (int c = 0; c < 16; c += 8) put_op8(A, row, col + c, a + c);
            written();
            if (threadIdx.x == 0) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) tc::mma_bf16(tmem, ak + 2 * ks, ak + 2 * ks, SM_IDESC_K, ks > 0);
                tc::commit(&bars->done);
            }
            take(v);
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = fmaf(pc, v[c], pb * a[c]);
#pragma unroll
            for (int c = 0; c < 16; c += 8) put_op8(A, row, col + c, v + c);
            const bool done = k + 1 == count;
            for (int s = 0; s < strips; ++s) {
                written();
                if (threadIdx.x == 0) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc::mma_bf16(tmem, ak + 2 * ks, xn + (uint64_t)(s * (SM_OP >> 4) + 128 * ks), SM_IDESC_MN, ks > 0);
                    tc::commit(&bars->done);
                }
                take(v);
                get_op8(X + s * SM_OP, row, col, a);
                get_op8(X + s * SM_OP, row, col + 8, a + 8);
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = fmaf(pa, a[c], v[c]);
                if (done) {
                    last(row, 64 * s + col, v);
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] *= 1.f / SP;
#pragma unroll
                    for (int c = 0; c < 16; c += 8) put_op8(X + s * SM_OP, row, col + c, v + c);
                }
            }
        }
    }
};

// sum over the block, in warp order
__device__ __forceinline__ double block_sum(double s, double* sm) {
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < SM_TPB / 32; ++w) s += sm[w];
    return s;
}

// One block per matrix, X [M][N] with M <= 64, N <= 256.  Thread t holds row t % 64 and every fourth group
// of 8 columns (a tall matrix: its rows are the columns of X); up to 64 columns stay in registers between
// the norm and the first split.
template <typename T, int PER_SM>
__global__ void __launch_bounds__(SM_TPB, PER_SM)
    small_kernel(const T* x, T* out, int M, int N, int tall, int steps, float ca, float cb, float cc, float eps, float scale) {
    extern __shared__ uint8_t raw[];
    Small m;
    const int strips = sm_strips(N), mn = M * N;
    m.begin(raw, strips);
    griddep_wait();
    griddep_launch();
    x += (long long)blockIdx.x * mn;
    out += (long long)blockIdx.x * mn;
    const int row = threadIdx.x & 63, c0 = (threadIdx.x >> 6) * 8;
    struct alignas(16) Lane {
        T v[16 / sizeof(T)];
    };
    constexpr int VEC = 16 / sizeof(T);
    const bool wide = !tall && N % VEC == 0 && mn % VEC == 0;  // 16-byte pieces of rows
    auto load8 = [&](int c, float (&v)[8]) {
        if (wide) {
#pragma unroll
            for (int h = 0; h < 8; h += VEC) {
                if (row < M && c + h < N) {
                    const Lane l = *reinterpret_cast<const Lane*>(x + row * N + c + h);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[h + e] = to_f(l.v[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[h + e] = 0.f;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = row < M && c + e < N ? to_f(x[tall ? (c + e) * M + row : row * N + c + e]) : 0.f;
        }
    };
    auto square = [](double s, const float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fma((double)v[e], (double)v[e], s);
        return s;
    };
    auto put = [&](int c, double inv, float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)((double)v[e] * inv);
        put_op8(m.X + (c >> 6) * SM_OP, row, c & 63, v);
    };
    if (strips == 1) {
        float v[2][8];
        load8(c0, v[0]);
        load8(c0 + 32, v[1]);
        const double s = square(0.0, v[0]) + square(0.0, v[1]);
        const double inv = inverse_norm(block_sum(s, m.bars->sums), eps) * SX;
        put(c0, inv, v[0]);
        put(c0 + 32, inv, v[1]);
    } else {
        double s = 0.0;
        float v[8];
#pragma unroll 4
        for (int c = c0; c < 64 * strips; c += 32) {
            load8(c, v);
            s = square(s, v);
        }
        const double inv = inverse_norm(block_sum(s, m.bars->sums), eps) * SX;
#pragma unroll 2
        for (int c = c0; c < 64 * strips; c += 32) {
            load8(c, v);
            put(c, inv, v);
        }
    }
    const float f = scale / (SX * SP);
    m.steps(strips, steps, ca, cb, cc, [&](int r, int c, const float (&v)[16]) {
        if (r >= M) return;
        if (wide) {
#pragma unroll
            for (int h = 0; h < 16; h += VEC)
                if (c + h < N) {
                    Lane l;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) l.v[e] = from_f<T>(v[h + e] * f);
                    *reinterpret_cast<Lane*>(out + r * N + c + h) = l;
                }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c + e < N) out[tall ? (c + e) * M + r : r * N + c + e] = from_f<T>(v[e] * f);
        }
    });
    m.end();
}

// ------------------------------------------------------------------ TTT-Linear, orthogonalised step
constexpr int D = 64, DD = D * D, ROWB = 128, TILE = TM * ROWB;

// G and C^T of one split of a unit's tokens, bf16, d <= 64 (the tensor maps fill up to 64 features with
// zeros): [V | K]^T K on the tcgen05 tensor cores.  Grid (S, U); part [U][S][2][64][64] (G, C^T).  Bound by HBM: K and V once (32 units of 3136 tokens: 10 us
// from cold caches, 384 of 196: 13).
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

// Four adjacent features of row `row` (of `rows`) of a [rows][d] tensor from feature c on, zero outside it.
// vec: d is a multiple of 4, so that they are one aligned load.
template <typename T>
__device__ __forceinline__ float4 load4(const T* base, int row, int rows, int c, int d, bool vec) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (row < rows) {
        const T* at = base + (long long)row * d + c;
        if (vec) {
            if (c < d) {
                struct alignas(4 * sizeof(T)) Lane {
                    T v[4];
                };
                const Lane l = *reinterpret_cast<const Lane*>(at);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = to_f(l.v[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < d) v[e] = to_f(at[e]);
        }
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void outer4(float (&acc)[4][4], float4 a, float4 b) {
    const float ax[4] = {a.x, a.y, a.z, a.w}, bx[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ax[i], bx[j], acc[i][j]);
}

// The same for any d <= 128 and type on the CUDA cores: grid (S, U, blocks of 64 x 64 of the d x d
// products), 256 threads with 4 x 4 values of G and of C each, 32 tokens at a time through shared memory,
// the next 32 on their way in registers.  part [U][S][2][pd][pd] (G, C^T), pd = 64 with zeros for d <= 64, d
// else.  Bound by the fp32 pipe; S fills the
// SMs (fp32 keeps its accuracy, which bf16 operands would not).  16 units of 4810 tokens, d = 64, fp32: 44 us
// from cold caches against 17 at that pipe's peak.
template <typename T>
__global__ void __launch_bounds__(256)
    gram_kernel(const T* __restrict__ k, const T* __restrict__ v, float* __restrict__ part, int N, int d, int pd) {
    constexpr int TOK = 32;
    __shared__ __align__(16) float tiles[3][TOK][68];  // K's rows of the product, K's and V's columns
    const int S = gridDim.x, r = blockIdx.x;
    const long long u = blockIdx.y;
    const int nb = (d + 63) / 64, i0 = blockIdx.z / nb * 64, j0 = blockIdx.z % nb * 64;
    const bool vec = d % 4 == 0, same = i0 == j0;
    griddep_wait();
    griddep_launch();
    const int per = (N + S - 1) / S, t0 = min(r * per, N), t1 = min(N, t0 + per);
    const T *ku = k + u * N * d, *vu = v + u * N * d;
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;  // also the place in a tile that a thread fills
    const int trow = threadIdx.x / 16;
    float4 next[3][2];
    auto fetch = [&](int t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            next[0][h] = load4(ku, t + trow + 16 * h, t1, i0 + tj, d, vec);
            if (!same) next[1][h] = load4(ku, t + trow + 16 * h, t1, j0 + tj, d, vec);
            next[2][h] = load4(vu, t + trow + 16 * h, t1, j0 + tj, d, vec);
        }
    };
    float g[4][4] = {}, c[4][4] = {};
    const int second = same ? 0 : 1;
    if (t0 < t1) fetch(t0);
    for (int t = t0; t < t1; t += TOK) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<float4*>(&tiles[0][trow + 16 * h][tj]) = next[0][h];
            if (!same) *reinterpret_cast<float4*>(&tiles[1][trow + 16 * h][tj]) = next[1][h];
            *reinterpret_cast<float4*>(&tiles[2][trow + 16 * h][tj]) = next[2][h];
        }
        __syncthreads();
        if (t + TOK < t1) fetch(t + TOK);
#pragma unroll 8
        for (int row = 0; row < TOK; ++row) {
            const float4 a = *reinterpret_cast<const float4*>(&tiles[0][row][ti]);
            outer4(g, a, *reinterpret_cast<const float4*>(&tiles[second][row][tj]));
            outer4(c, a, *reinterpret_cast<const float4*>(&tiles[2][row][tj]));
        }
        __syncthreads();
    }
    float* p = part + (u * S + r) * 2 * pd * pd;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = i0 + ti + i, col = j0 + tj + j;
            if (row < pd && col < pd) {
                p[(long long)row * pd + col] = g[i][j];
                p[(long long)pd * pd + (long long)col * pd + row] = c[i][j];
            }
        }
}

// One block per unit, d <= 64: the partials are added in split order, g = (1/N)(G W0 - C) is formed in
// fp32 on the CUDA cores (4 x 4 values a thread), orthogonalised, and W* = W0 - eta U written, to w_star
// [U][d][d] and, filled up with zeros, to w_pad [U][64][64] (either may be null).  The partials are 64 x 64.
constexpr int FLD = D + 4;
constexpr int update_smem_bytes() { return small_smem_bytes(D); }
template <int PER_SM>
__global__ void __launch_bounds__(SM_TPB, PER_SM)
    update_kernel(const float* __restrict__ part, const float* __restrict__ w0, float* __restrict__ w_star,
                  float* __restrict__ w_pad, int S, int H, int d, float inv_n, float eta, int steps, float ca, float cb, float cc, float eps) {
    extern __shared__ uint8_t raw[];
    Small m;
    m.begin(raw, 1);
    // G and W0 [k][64 + 4] before the steps, where X, A and the exchange go
    float *G = reinterpret_cast<float*>(m.X), *W = G + D * FLD;
    static_assert(2 * D * FLD * 4 <= 2 * SM_OP + SM_EX, "G and W0 fit");
    const long long u = blockIdx.x;
    const int dd = d * d, tid = threadIdx.x;
    w0 += (u % H) * dd;
    griddep_wait();  // the partials; W0 too may be new
    griddep_launch();
    if (d == D) {
#pragma unroll
        for (int i = 0; i < DD / 4 / SM_TPB; ++i) {
            const int e = (tid + i * SM_TPB) * 4;
            *reinterpret_cast<float4*>(W + (e / D) * FLD + e % D) = __ldg(reinterpret_cast<const float4*>(w0 + e));
        }
    } else {
        for (int e = tid; e < DD; e += SM_TPB) {
            const int r = e / D, c = e % D;
            W[r * FLD + c] = r < d && c < d ? __ldg(w0 + r * d + c) : 0.f;
        }
    }
    part += u * S * 2 * DD;
    const int tr = (tid >> 4) * 4, tc = (tid & 15) * 4;  // rows tr .. + 3, columns tc .. + 3
    float acc[4][4];  // -C first, from C^T
    // G (symmetric: rows are its k) and C^T, a split's loads all in flight
    float4 g4[4], c4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g4[i] = c4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int q = 0; q < S; ++q) {
        const float4* p4 = reinterpret_cast<const float4*>(part + (size_t)q * 2 * DD);
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __ldg(p4 + tid + i * SM_TPB);
            y[i] = __ldg(p4 + (DD + (tc + i) * D + tr) / 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g4[i].x += x[i].x, g4[i].y += x[i].y, g4[i].z += x[i].z, g4[i].w += x[i].w;
            c4[i].x += y[i].x, c4[i].y += y[i].y, c4[i].z += y[i].z, c4[i].w += y[i].w;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = (tid + i * SM_TPB) * 4;
        *reinterpret_cast<float4*>(G + (e / D) * FLD + e % D) = g4[i];
        acc[0][i] = -c4[i].x, acc[1][i] = -c4[i].y, acc[2][i] = -c4[i].z, acc[3][i] = -c4[i].w;
    }
    __syncthreads();
    float gw[4][4] = {};
#pragma unroll 8
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
    const double inv = inverse_norm(block_sum(s, m.bars->sums), eps) * SX;  // its barrier: G and W0 have been read
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v[4] = {(float)(acc[i][0] * inv), (float)(acc[i][1] * inv), (float)(acc[i][2] * inv), (float)(acc[i][3] * inv)};
        uint2 hi, lo;
        split4(v, hi, lo);
        uint8_t* at = m.X + swz<3>((uint32_t)(tr + i) * 128 + (uint32_t)tc * 2);
        *reinterpret_cast<uint2*>(at) = hi;
        *reinterpret_cast<uint2*>(at + SM_M * 128) = lo;
    }
    m.steps(1, steps, ca, cb, cc, [&](int r, int c, const float (&v)[16]) {
        const float f = -eta / (SX * SP);
        if (d == D) {
            float* to = (w_star ? w_star : w_pad) + u * DD + r * D + c;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 w = __ldg(reinterpret_cast<const float4*>(w0 + r * D + c + e));
                *reinterpret_cast<float4*>(to + e) =
                    make_float4(fmaf(f, v[e], w.x), fmaf(f, v[e + 1], w.y), fmaf(f, v[e + 2], w.z), fmaf(f, v[e + 3], w.w));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const bool in = r < d && c + e < d;
                const float w = in ? fmaf(f, v[e], __ldg(w0 + r * d + c + e)) : 0.f;
                if (in && w_star) w_star[u * dd + r * d + c + e] = w;
                if (w_pad) w_pad[u * DD + r * D + c + e] = w;
            }
        }
    });
    m.end();
}

// O = Q W on the CUDA cores for any d <= 128 and type: 64 tokens x 64 output features per block, 4 x 4
// values a thread, 64 input features at a time through shared memory (both operands read four features of
// k at a time: eight 16-byte reads for 64 multiply-adds).  Grid (token tiles, U, feature tiles).  16 units of
// 4810 tokens, d = 64, fp32: 24 us from cold caches against 9 at the fp32 pipe's peak.
template <typename T>
__global__ void __launch_bounds__(256)
    apply_kernel(const T* __restrict__ q, const float* __restrict__ w, T* __restrict__ out, int N, int d) {
    __shared__ __align__(16) float qs[64][68], ws[64][68];  // [token][k], [k][feature]
    const long long u = blockIdx.y;
    const int t0 = blockIdx.x * 64, j0 = blockIdx.z * 64;
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4, row = threadIdx.x / 16;
    const bool vec = d % 4 == 0;
    griddep_wait();
    griddep_launch();
    const T* qu = q + u * N * d;
    const float* wu = w + u * d * d;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < d; k0 += 64) {
        float4 a[4], b[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            a[h] = load4(qu, t0 + row + 16 * h, N, k0 + tj, d, vec);
            b[h] = load4(wu, k0 + row + 16 * h, d, j0 + tj, d, vec);
        }
        if (k0 > 0) __syncthreads();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            *reinterpret_cast<float4*>(&qs[row + 16 * h][tj]) = a[h];
            *reinterpret_cast<float4*>(&ws[row + 16 * h][tj]) = b[h];
        }
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < 64; k += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = *reinterpret_cast<const float4*>(&qs[ti + i][k]);
                y[i] = *reinterpret_cast<const float4*>(&ws[k + i][tj]);
            }
            outer4(acc, make_float4(x[0].x, x[1].x, x[2].x, x[3].x), y[0]);
            outer4(acc, make_float4(x[0].y, x[1].y, x[2].y, x[3].y), y[1]);
            outer4(acc, make_float4(x[0].z, x[1].z, x[2].z, x[3].z), y[2]);
            outer4(acc, make_float4(x[0].w, x[1].w, x[2].w, x[3].w), y[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + ti + i;
        if (t >= N) break;
        T* o = out + (u * N + t) * d + j0 + tj;
        if (vec) {
            struct alignas(4 * sizeof(T)) Lane {
                T v[4];
            } l;
#pragma unroll
            for (int e = 0; e < 4; ++e) l.v[e] = from_f<T>(acc[i][e]);
            if (j0 + tj < d) *reinterpret_cast<Lane*>(o) = l;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j0 + tj + e < d) o[e] = from_f<T>(acc[i][e]);
        }
    }
}

// ---- d > 64: the steps of the general path between these two
// The S partials of a unit added in split order, into the first
__global__ void __launch_bounds__(TPB) fold_kernel(float* __restrict__ part, int S, int dd2) {
    float* p = part + (long long)blockIdx.x * S * dd2;
    const int e = blockIdx.y * TPB + threadIdx.x;
    griddep_wait();
    griddep_launch();
    if (e >= dd2) return;
    float s = p[e];
#pragma unroll 8
    for (int q = 1; q < S; ++q) s += p[(long long)q * dd2 + e];
    p[e] = s;
}

// g[u] = (1/N)(G W0[h] - C) from the folded partials, which lie S apart
__global__ void __launch_bounds__(TPB)
    gradient_kernel(const float* __restrict__ part, const float* __restrict__ w0, float* __restrict__ g, int S, int H, int d,
                    float inv_n) {
    const long long u = blockIdx.x;
    const int dd = d * d, e = blockIdx.y * TPB + threadIdx.x;
    griddep_wait();
    griddep_launch();
    if (e >= dd) return;
    const int i = e / d, j = e % d;
    const float *W0 = w0 + (u % H) * dd, *G = part + u * S * 2 * dd;
    float gw = 0.f;
#pragma unroll 8
    for (int m = 0; m < d; ++m) gw = fmaf(G[i * d + m], W0[m * d + j], gw);
    g[u * dd + e] = (gw - G[dd + j * d + i]) * inv_n;
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

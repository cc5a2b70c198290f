// norm.cuh -- layer norm over the feature axis of token rows, forward and backward.
//
// The norm in front of the TTT block ("ViT^3" blog: the block wrapper is Norm -> TTT block ->
// Residual).  Per row x in R^C with weight g and bias b:
//     mu = mean(x),  r = 1 / sqrt(mean((x - mu)^2) + eps),  xh = (x - mu) r,  y = xh g + b,
// and for an upstream gradient dy, with t = dy g:
//     dx = r (t - mean(t) - xh mean(t xh)),   dg = sum over rows of dy xh,   db = sum of dy.
//
// A row is held in registers by a group of threads (part of a warp, a warp, or several warps),
// so x and dy are read from memory once.  Statistics take two rounds of reductions: mu first,
// then with c = x - mu the sums of c and c^2 (backward: also of t and t c).  The mean of c is
// what rounding left in mu; taking it out again (xh = (c - mean(c)) r, variance = mean(c^2) -
// mean(c)^2) keeps rows exact whose offset is large against their spread.  All sums are fp32.
#pragma once
#include "common.cuh"

namespace lnorm {

constexpr int THREADS = 256;    // threads of a block with rows of up to 8 warps; wider rows take one block each
constexpr int MAX_EPT = 16;     // elements of a row that one thread holds at most
constexpr int MAX_COLS = 1024 * MAX_EPT;

template <typename T, int VEC>
struct Pack;
template <>
struct Pack<float, 1> {
    static __device__ __forceinline__ void load(const float* p, float* v) { v[0] = *p; }
    static __device__ __forceinline__ void store(float* p, const float* v) { *p = v[0]; }
};
template <>
struct Pack<float, 4> {
    static __device__ __forceinline__ void load(const float* p, float* v) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* v) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Pack<__nv_bfloat16, 1> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* v) { v[0] = __bfloat162float(*p); }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) { *p = __float2bfloat16_rn(v[0]); }
};
template <>
struct Pack<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* v) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                  pack_bf16(v[6], v[7]));
    }
};

// How a block is split over rows: `lanes` threads of a warp (a power of two) times `warps` warps
// hold one row (warps > 1 only with lanes = 32).
struct Shape {
    int lanes, warps, threads;
    __host__ __device__ int rows_per_block() const { return threads / (lanes * warps); }
};

// Sum of K values over the threads of one row.  Within a warp by exchange; across warps through
// `red` ([2][K][32], `which` alternates so that one barrier per round is enough), in warp order.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], const Shape s, float* red, int which) {
    for (int o = s.lanes >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (s.warps == 1) return;
    const int warp = threadIdx.x >> 5, first = warp / s.warps * s.warps;
    float* r = red + which * K * 32;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) r[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = 0.f;
        for (int w = 0; w < s.warps; ++w) v[k] += r[k * 32 + first + w];
    }
}

// ----------------------------------------------------------------------------- forward ---
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024)
    forward_kernel(const T* x, const float* __restrict__ gamma, const float* __restrict__ beta, T* y, int rows, int C,
                   float eps, float inv_c, const Shape s) {
    __shared__ float red[2 * 2 * 32];
    const int tpr = s.lanes * s.warps, rpb = s.rows_per_block();
    const int at = threadIdx.x % tpr;
    const long long row = (long long)blockIdx.x * rpb + threadIdx.x / tpr;
    const bool live = row < rows;
    const long long base = row * C;
    float v[NV][VEC];
    float s1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (at + i * tpr) * VEC;
        if (live && c < C)
            Pack<T, VEC>::load(x + base + c, v[i]);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s1[0] += v[i][e];
    }
    row_sum<1>(s1, s, red, 0);
    const float mean = s1[0] * inv_c;
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool in = (at + i * tpr) * VEC < C;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            v[i][e] -= mean;
            if (in) {
                s2[0] += v[i][e];
                s2[1] = fmaf(v[i][e], v[i][e], s2[1]);
            }
        }
    }
    row_sum<2>(s2, s, red + 64, 0);
    const float off = s2[0] * inv_c;
    const float rstd = rsqrtf(fmaxf(s2[1] * inv_c - off * off, 0.f) + eps);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (at + i * tpr) * VEC;
        if (c >= C) continue;
        float g[VEC], o[VEC];
        if constexpr (VEC == 8) {
            Pack<float, 4>::load(gamma + c, g);
            Pack<float, 4>::load(gamma + c + 4, g + 4);
        } else {
            Pack<float, VEC>::load(gamma + c, g);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = (v[i][e] - off) * rstd * g[e];
        if (beta)
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] += __ldg(beta + c + e);
        Pack<T, VEC>::store(y + base + c, o);
    }
}

// ----------------------------------------------------------------------------- backward --
// Each group of threads walks rows `group, group + groups, ...` and keeps its columns' sums of
// dy xh and dy in registers; the block adds its groups' sums in order and writes one partial row
// of each per block, part[block][2][C].
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024)
    backward_kernel(const T* dy, const T* x, const float* __restrict__ gamma, T* dx, float* __restrict__ part, int rows,
                    int C, float eps, float inv_c, const Shape s) {
    extern __shared__ float sums[];  // [rows_per_block][2][C] when a block holds several rows
    __shared__ float red[2 * 32 + 2 * 4 * 32];
    const int tpr = s.lanes * s.warps, rpb = s.rows_per_block();
    const int at = threadIdx.x % tpr, grp = threadIdx.x / tpr;
    float g[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (at + i * tpr) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            g[i][e] = c < C ? __ldg(gamma + c + e) : 0.f;
            dg[i][e] = db[i][e] = 0.f;
        }
    }
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * rpb; r0 < rows; r0 += (long long)gridDim.x * rpb, turn ^= 1) {
        const long long row = r0 + grp, base = row * C;
        const bool live = row < rows;
        float v[NV][VEC], t[NV][VEC];
        float s1[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (at + i * tpr) * VEC;
            if (live && c < C) {
                Pack<T, VEC>::load(x + base + c, v[i]);
                Pack<T, VEC>::load(dy + base + c, t[i]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] = t[i][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) s1[0] += v[i][e];
        }
        row_sum<1>(s1, s, red, turn);
        const float mean = s1[0] * inv_c;
        float s4[4] = {0.f, 0.f, 0.f, 0.f};  // c, c^2, t, t c
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = (at + i * tpr) * VEC < C;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[i][e] = in ? v[i][e] - mean : 0.f;
                const float tg = t[i][e] * g[i][e];
                s4[0] += v[i][e];
                s4[1] = fmaf(v[i][e], v[i][e], s4[1]);
                s4[2] += tg;
                s4[3] = fmaf(tg, v[i][e], s4[3]);
            }
        }
        row_sum<4>(s4, s, red + 64, turn);
        const float off = s4[0] * inv_c;
        const float rstd = rsqrtf(fmaxf(s4[1] * inv_c - off * off, 0.f) + eps);
        const float mt = s4[2] * inv_c;
        const float mtx = (s4[3] * inv_c - off * mt) * rstd;  // mean(t xh)
        if (live)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (at + i * tpr) * VEC;
                if (c >= C) continue;
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (v[i][e] - off) * rstd;
                    o[e] = rstd * (fmaf(t[i][e], g[i][e], -mt) - xh * mtx);
                    dg[i][e] = fmaf(t[i][e], xh, dg[i][e]);
                    db[i][e] += t[i][e];
                }
                Pack<T, VEC>::store(dx + base + c, o);
            }
    }
    float* p = part + (long long)blockIdx.x * 2 * C;
    if (rpb > 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (at + i * tpr) * VEC;
            if (c >= C) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                sums[grp * 2 * C + c + e] = dg[i][e];
                sums[grp * 2 * C + C + c + e] = db[i][e];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * C; c += blockDim.x) {
            float a = 0.f;
            for (int r = 0; r < rpb; ++r) a += sums[r * 2 * C + c];
            p[c] = a;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (at + i * tpr) * VEC;
            if (c >= C) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                p[c + e] = dg[i][e];
                p[C + c + e] = db[i][e];
            }
        }
    }
}

// dg, db = the partials' sums over the blocks, in block order within each of 8 strands, the
// strands then in order.  32 columns x 8 strands per block.
__global__ void __launch_bounds__(256)
    finish_kernel(const float* __restrict__ part, float* __restrict__ dgamma, float* __restrict__ dbeta, int blocks,
                  int C) {
    __shared__ float sm[8][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), strand = threadIdx.x >> 5;
    float a = 0.f;
    if (col < 2 * C)
        for (int b = strand; b < blocks; b += 8) a += part[(long long)b * 2 * C + col];
    sm[strand][threadIdx.x & 31] = a;
    __syncthreads();
    if (strand == 0 && col < 2 * C) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += sm[w][threadIdx.x & 31];
        if (col < C)
            dgamma[col] = t;
        else if (dbeta)
            dbeta[col - C] = t;
    }
}

}  // namespace lnorm

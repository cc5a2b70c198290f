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
constexpr int THREADS_BWD = 512;  // of the backward pass, one block an SM (half the partial sums of two blocks of 256)
constexpr int MAX_EPT = 16;     // elements of a row that one thread holds at most
constexpr int MAX_COLS = 1024 * MAX_EPT;
constexpr int STRANDS = 32;     // of the sum over blocks

// VEC adjacent elements as they lie in memory
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
    __device__ __forceinline__ void get(float* f) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = to_f(v[e]);
    }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = from_f<T>(f[e]);
    }
};
template <int VEC>
__device__ __forceinline__ void get_weights(const float* w, float* f) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(w + e));
            f[e] = x.x, f[e + 1] = x.y, f[e + 2] = x.z, f[e + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = __ldg(w + e);
    }
}

// How a block is split over rows: `lanes` threads of a warp (a power of two) times `warps` warps
// hold one row (warps > 1 only with lanes = 32).
struct Shape {
    int lanes, warps, threads;
    __host__ __device__ int rows_per_block() const { return threads / (lanes * warps); }
};

// Sums of K values over the threads of one row.  Within a warp by exchange; across warps through
// `red` ([K][32]), in warp order.  Buffers of successive rounds have to differ.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], const Shape s, float* red) {
    for (int o = s.lanes >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (s.warps == 1) return;
    const int warp = threadIdx.x >> 5, first = warp / s.warps * s.warps;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) red[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = 0.f;
        for (int w = 0; w < s.warps; ++w) v[k] += red[k * 32 + first + w];
    }
}

// ----------------------------------------------------------------------------- forward ---
// A group of threads takes FLY rows at once: their loads are in flight together, and weight and bias
// are read once for all of them.  Bound by HBM (and the launch when small): 100352 x 64 bf16 in 6.8 us,
// 3.8 TB/s (25600 x 192 fp32 5.5 TB/s); 196 x 384 bf16 in 2.2 us.
template <typename T, int VEC, int NV, int FLY, int MAXT>
__global__ void __launch_bounds__(MAXT)
    forward_kernel(const T* x, const float* __restrict__ gamma, const float* __restrict__ beta, T* y, int rows, int C,
                   float eps, float inv_c, const Shape s) {
    using L = Pack<T, VEC>;
    __shared__ float red[3 * FLY * 32];
    const int tpr = s.lanes * s.warps, rpb = s.rows_per_block();
    const int at = threadIdx.x % tpr;
    const long long row0 = (long long)blockIdx.x * rpb * FLY + threadIdx.x / tpr;
    griddep_wait();
    griddep_launch();
    float v[FLY][NV][VEC];
    float s1[FLY];
    L raw[FLY][NV];
#pragma unroll
    for (int f = 0; f < FLY; ++f)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const long long row = row0 + f * rpb;
            const int c = (at + i * tpr) * VEC;
            if (row < rows && c < C) raw[f][i] = *reinterpret_cast<const L*>(x + row * C + c);
        }
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
        s1[f] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (row0 + f * rpb < rows && (at + i * tpr) * VEC < C)
                raw[f][i].get(v[f][i]);
            else
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[f][i][e] = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) s1[f] += v[f][i][e];
        }
    }
    row_sum<FLY>(s1, s, red);
    float s2[2 * FLY];
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
        const float mean = s1[f] * inv_c;
        s2[2 * f] = s2[2 * f + 1] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = (at + i * tpr) * VEC < C;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[f][i][e] = in ? v[f][i][e] - mean : 0.f;
                s2[2 * f] += v[f][i][e];
                s2[2 * f + 1] = fmaf(v[f][i][e], v[f][i][e], s2[2 * f + 1]);
            }
        }
    }
    row_sum<2 * FLY>(s2, s, red + FLY * 32);
    float off[FLY], rstd[FLY];
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
        off[f] = s2[2 * f] * inv_c;
        rstd[f] = rsqrtf(fmaxf(s2[2 * f + 1] * inv_c - off[f] * off[f], 0.f) + eps);
        if (s2[2 * f + 1] != s2[2 * f + 1]) rstd[f] = s2[2 * f + 1];  // a NaN is not clamped away
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (at + i * tpr) * VEC;
        if (c >= C) continue;
        float g[VEC], b[VEC];
        get_weights<VEC>(gamma + c, g);
        if (beta)
            get_weights<VEC>(beta + c, b);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) b[e] = 0.f;
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
            if (row0 + f * rpb >= rows) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = fmaf((v[f][i][e] - off[f]) * rstd[f], g[e], b[e]);
            L out;
            out.set(o);
            *reinterpret_cast<L*>(y + (row0 + f * rpb) * C + c) = out;
        }
    }
}

// ----------------------------------------------------------------------------- backward --
// Each group of threads walks rows `group, group + groups, ...` and keeps its columns' sums of dy xh
// and dy in registers; the block adds its groups' sums in order and writes one partial row of each,
// part[block][2][C].  The next DEPTH - 1 rows are on their way into shared memory by asynchronous copies,
// each thread fetching what it will read itself (no barrier); 2-byte loads and the widest rows, which have
// no such copies or no room, keep one row ahead in registers.  12544 x 384 bf16 in 14.1 us with the second
// kernel (one row ahead in registers and two blocks of 256 an SM: 16.7); long inputs run at 4.4 TB/s.
// Rows above 8192 take 1024 threads of 64 registers, which spill 590 to 770 bytes a thread: 1500 x 8192 bf16 in 36 us, 1500
// x 8200 in 109, 1500 x 16384 in 192 (fp32 223, 16383 columns 317).
template <typename T, int VEC, int NV, int MAXT>
struct Ahead {
    static constexpr int BYTES = NV * VEC * (int)sizeof(T);  // of a thread, per tensor and row
    static constexpr bool ASYNC = VEC * sizeof(T) >= 4 && MAXT <= 512;
    static constexpr int DEPTH = BYTES <= 48 ? 4 : 3;
    static constexpr int smem(int threads) { return ASYNC ? DEPTH * 2 * BYTES * threads : 0; }
};
__device__ __forceinline__ void copy_ahead(uint32_t to, const void* from, int bytes) {
    if (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

template <typename T, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == THREADS ? 2 : 1)
    backward_kernel(const T* dy, const T* x, const float* __restrict__ gamma, T* dx, float* __restrict__ part, int rows,
                    int C, float eps, float inv_c, const Shape s) {
    using L = Pack<T, VEC>;
    using A = Ahead<T, VEC, NV, MAXT>;
    extern __shared__ __align__(16) uint8_t smem[];  // rows on their way; then [rows_per_block][2][C] sums
    float* sums = reinterpret_cast<float*>(smem);
    __shared__ float red[2][5 * 32];
    const int tpr = s.lanes * s.warps, rpb = s.rows_per_block();
    const int at = threadIdx.x % tpr, grp = threadIdx.x / tpr;
    griddep_wait();
    griddep_launch();
    L rx[NV], rt[NV];
    // [slot][tensor][vector][thread]
    auto place = [&](int slot, int tensor, int i) { return ((slot * 2 + tensor) * NV + i) * s.threads + (int)threadIdx.x; };
    auto fetch = [&](long long row, int slot) {
        if (row < rows)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (at + i * tpr) * VEC;
                if (c >= C) continue;
                if constexpr (A::ASYNC) {
                    copy_ahead(smem_u32(smem) + place(slot, 0, i) * (uint32_t)sizeof(L), x + row * C + c, sizeof(L));
                    copy_ahead(smem_u32(smem) + place(slot, 1, i) * (uint32_t)sizeof(L), dy + row * C + c, sizeof(L));
                } else {
                    rx[i] = *reinterpret_cast<const L*>(x + row * C + c);
                    rt[i] = *reinterpret_cast<const L*>(dy + row * C + c);
                }
            }
        if constexpr (A::ASYNC) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const long long stride = (long long)gridDim.x * rpb;
    long long r0 = (long long)blockIdx.x * rpb;
    if constexpr (A::ASYNC) {
#pragma unroll
        for (int d = 0; d < A::DEPTH - 1; ++d) fetch(r0 + grp + d * stride, d);
    } else {
        fetch(r0 + grp, 0);
    }
    int slot = 0;
    float g[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (at + i * tpr) * VEC;
        if (c < C)
            get_weights<VEC>(gamma + c, g[i]);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[i][e] = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) dg[i][e] = db[i][e] = 0.f;
    }
    for (int turn = 0; r0 < rows; r0 += stride, turn ^= 1) {
        const long long row = r0 + grp;
        const bool live = row < rows;
        float v[NV][VEC], t[NV][VEC];
        float s1[1] = {0.f};
        if constexpr (A::ASYNC) {
            // the slot freed by the last row takes the row DEPTH - 1 ahead; then this row's copies are over
            fetch(row + (A::DEPTH - 1) * stride, slot == 0 ? A::DEPTH - 1 : slot - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(A::DEPTH - 1) : "memory");
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                rx[i] = reinterpret_cast<const L*>(smem)[place(slot, 0, i)];
                rt[i] = reinterpret_cast<const L*>(smem)[place(slot, 1, i)];
            }
            slot = slot + 1 == A::DEPTH ? 0 : slot + 1;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (live && (at + i * tpr) * VEC < C) {
                rx[i].get(v[i]);
                rt[i].get(t[i]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] = t[i][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) s1[0] += v[i][e];
        }
        if constexpr (!A::ASYNC) fetch(row + stride, 0);
        row_sum<1>(s1, s, red[turn]);
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
        row_sum<4>(s4, s, red[turn] + 32);
        const float off = s4[0] * inv_c;
        float rstd = rsqrtf(fmaxf(s4[1] * inv_c - off * off, 0.f) + eps);
        if (s4[1] != s4[1]) rstd = s4[1];  // a NaN is not clamped away
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
                L out;
                out.set(o);
                *reinterpret_cast<L*>(dx + row * C + c) = out;
            }
    }
    float* p = part + (long long)blockIdx.x * 2 * C;
    auto put = [&](float* to, const float (&v)[NV][VEC]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (at + i * tpr) * VEC;
            if (c >= C) continue;
            if constexpr (VEC % 4 == 0) {
#pragma unroll
                for (int e = 0; e < VEC; e += 4)
                    *reinterpret_cast<float4*>(to + c + e) = make_float4(v[i][e], v[i][e + 1], v[i][e + 2], v[i][e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) to[c + e] = v[i][e];
            }
        }
    };
    if (rpb > 1) {
        if constexpr (A::ASYNC) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();  // every thread has read its last row: the sums may go over them
        }
        put(sums + grp * 2 * C, dg);
        put(sums + grp * 2 * C + C, db);
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * C; c += blockDim.x) {
            float a = 0.f;
#pragma unroll 8
            for (int r = 0; r < rpb; ++r) a += sums[r * 2 * C + c];
            p[c] = a;
        }
    } else {
        put(p, dg);
        put(p + C, db);
    }
}

// dg, db = the partials' sums over the blocks: 32 columns x 32 strands per block, a strand adding every
// 32nd partial in order (their loads in flight together), the strands then added in order.
__global__ void __launch_bounds__(32 * STRANDS)
    finish_kernel(const float* __restrict__ part, float* __restrict__ dgamma, float* __restrict__ dbeta, int blocks,
                  int C) {
    __shared__ float sm[STRANDS][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), strand = threadIdx.x >> 5;
    griddep_wait();
    griddep_launch();
    float a = 0.f;
    if (col < 2 * C)
#pragma unroll 5
        for (int b = strand; b < blocks; b += STRANDS) a += part[(long long)b * 2 * C + col];
    sm[strand][threadIdx.x & 31] = a;
    __syncthreads();
    if (strand == 0 && col < 2 * C) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < STRANDS; ++w) t += sm[w][threadIdx.x];
        if (col < C)
            dgamma[col] = t;
        else if (dbeta)
            dbeta[col - C] = t;
    }
}

}  // namespace lnorm

// orth.cuh -- the orthogonal factor of an update by Newton-Schulz products.
//
// X_0 = X / max(|X|_F, eps), then `steps` times
//     A = X X^T,   B = b A + c A^2,   X <- a X + B X,
// which sends every singular value s of X_0 to p(s) = a s + b s^3 + c s^5 and leaves its singular
// vectors.  Everything is done on the side that is shorter (X is taken transposed when it is
// tall).  Sums of squares are formed in fp64, so that no finite X overflows its norm.
#pragma once
#include "common.cuh"

namespace orth {

constexpr int TPB = 256;
constexpr int MAX_PARTS = 64;

// part[u][p] = sum of squares of piece p of matrix u
template <typename T>
__global__ void __launch_bounds__(TPB) square_kernel(const T* __restrict__ x, double* __restrict__ part, long long mn) {
    __shared__ double sm[TPB / 32];
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

// y[u][i][j] = x / max(norm, eps), [M][N] with M <= N (transposed on the way when tall)
template <typename T>
__global__ void __launch_bounds__(TPB)
    start_kernel(const T* __restrict__ x, const double* __restrict__ part, float* __restrict__ y, int parts, int M,
                 int N, int tall, float eps) {
    double s = 0.0;
    for (int p = 0; p < parts; ++p) s += part[(long long)blockIdx.y * parts + p];
    const double inv = 1.0 / fmax(sqrt(s), (double)eps);
    const long long mn = (long long)M * N, i = (long long)blockIdx.x * TPB + threadIdx.x;
    if (i >= mn) return;
    const long long from = tall ? (i % N) * M + i / N : i;
    y[blockIdx.y * mn + i] = (float)((double)to_f(x[blockIdx.y * mn + from]) * inv);
}

// C = alpha A B' + beta D per matrix, fp32; A [M][K], B' = B [K][N] or B^T with B [N][K]
__global__ void __launch_bounds__(TPB)
    product_kernel(const float* __restrict__ a, const float* __restrict__ b, const float* __restrict__ d,
                   float* __restrict__ c, int M, int N, int K, int trans_b, float alpha, float beta) {
    __shared__ float As[16][65], Bs[16][65];
    const long long u = blockIdx.z;
    a += u * M * K;
    b += u * N * K;
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int e = threadIdx.x; e < 1024; e += TPB) {
            const int i = e / 16, k = e % 16;
            As[k][i] = i0 + i < M && k0 + k < K ? a[(long long)(i0 + i) * K + k0 + k] : 0.f;
            if (trans_b) {
                Bs[k][i] = j0 + i < N && k0 + k < K ? b[(long long)(j0 + i) * K + k0 + k] : 0.f;
            } else {
                const int kk = e / 64, j = e % 64;
                Bs[kk][j] = j0 + j < N && k0 + kk < K ? b[(long long)(k0 + kk) * N + j0 + j] : 0.f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][ti + i], Bs[k][tj + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (i0 + ti + i < M && j0 + tj + j < N) {
                const long long e = u * M * N + (long long)(i0 + ti + i) * N + j0 + tj + j;
                c[e] = alpha * acc[i][j] + (d ? beta * d[e] : 0.f);
            }
}

// out = scale y (+ base, which lies [rows of `share` matrices]), transposed back when tall
template <typename T>
__global__ void __launch_bounds__(TPB)
    end_kernel(const float* __restrict__ y, T* __restrict__ out, int M, int N, int tall, float scale) {
    const long long mn = (long long)M * N, i = (long long)blockIdx.x * TPB + threadIdx.x;
    if (i >= mn) return;
    const long long from = tall ? (i % M) * N + i / M : i;
    out[blockIdx.y * mn + i] = from_f<T>(scale * y[blockIdx.y * mn + from]);
}

// ------------------------------------------------- the TTT-Linear step with such an update ---
// g[u] = (1/N)(G W0[h] - C) from gc[u] = [G | C]
__global__ void __launch_bounds__(TPB)
    gradient_kernel(const float* __restrict__ gc, const float* __restrict__ w0, float* __restrict__ g, int H, int d,
                    float inv_n) {
    const long long u = blockIdx.x;
    const int e = blockIdx.y * TPB + threadIdx.x;
    if (e >= d * d) return;
    const int i = e / d, j = e % d;
    const float* G = gc + u * 2 * d * d + (long long)i * 2 * d;
    const float* W0 = w0 + (u % H) * d * d;
    float s = 0.f;
    for (int m = 0; m < d; ++m) s = fmaf(G[m], W0[m * d + j], s);
    g[u * d * d + e] = (s - G[d + j]) * inv_n;
}

// W* = W0[h] - eta U
__global__ void __launch_bounds__(TPB)
    step_kernel(const float* __restrict__ upd, const float* __restrict__ w0, float* __restrict__ wst,
                float* __restrict__ w_star_out, int H, int dd, float eta) {
    const long long u = blockIdx.x;
    const int e = blockIdx.y * TPB + threadIdx.x;
    if (e >= dd) return;
    const float w = w0[(u % H) * dd + e] - eta * upd[u * dd + e];
    wst[u * dd + e] = w;
    if (w_star_out) w_star_out[u * dd + e] = w;
}

}  // namespace orth

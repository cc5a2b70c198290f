// rope.cuh -- rotary positions with several axes (row and column of an image's token grid; time
// as well for video), applied to Q and K ahead of the TTT layer.
//
// The first dims[0] features of a head turn with the token's position on axis 0, the next dims[1]
// with axis 1, and so on; what is left of the head passes unchanged.  Axis a of width s has s/2
// pairs, pair j turning by  angle = p_a base^(-2 j / s):
//     (x, y) -> (x cos - y sin, y cos + x sin).
// A pair is (j, j + s/2) of the axis' section, or (2j, 2j + 1) when interleaved.  A rotation's
// transpose is its inverse, so the backward pass is the same kernel with sin negated.
//
// Angles of far positions need more than 32 bits: the position times the frequency in turns
// (theta / 2 pi) is formed and reduced to [-1/2, 1/2] in fp64, then sincospi in fp32 of that
// fraction (error about 1e-7).  A block does this once per (token, pair) of its token tile and
// keeps the table in shared memory for all its heads and both tensors.
#pragma once
#include "common.cuh"

namespace rope {

constexpr int THREADS = 256;
constexpr int MAX_AXES = 4;
constexpr int MAX_D = 512;

struct Axes {
    int n;                 // axes
    int at[MAX_AXES];      // first feature of the section
    int dims[MAX_AXES];    // its width
    int grid[MAX_AXES];    // the token grid, when positions are not given
    int pairs;             // all pairs
};
struct View {              // element strides; the features of a head are adjacent
    long long b, h, n;
};
struct Params {
    const float* pos;      // [N][axes] or [B][N][axes], or null: the grid in raster order
    long long pos_b;       // stride of a batch entry, 0 when shared
    int B, H, N, d, TN;
    int interleaved;
    float sign;            // -1: inverse
    Axes ax;
    View qi, ki, qo, ko;
    double turns[MAX_D / 2];  // frequency of each pair / 2 pi
};

template <typename T>
__global__ void __launch_bounds__(THREADS)
    rope_kernel(const T* q, const T* k, T* qout, T* kout, const __grid_constant__ Params p) {
    extern __shared__ float2 table[];  // [TN][pairs]: cos, sin
    const int t0 = blockIdx.x * p.TN, tn = min(p.TN, p.N - t0);
    const int b = blockIdx.z, P = p.ax.pairs;
    for (int i = threadIdx.x; i < tn * P; i += THREADS) {
        const int t = i / P, j = i % P, tok = t0 + t;
        int a = 0;
        while (a + 1 < p.ax.n && 2 * j >= p.ax.at[a + 1]) ++a;
        double x;
        if (p.pos) {
            x = (double)p.pos[b * p.pos_b + (long long)tok * p.ax.n + a];
        } else {
            int cell = tok;
            for (int c = p.ax.n - 1; c > a; --c) cell /= p.ax.grid[c];
            x = (double)(cell % p.ax.grid[a]);
        }
        double r = x * p.turns[j];
        r -= rint(r);
        float sn, cs;
        sincospif(2.f * (float)r, &sn, &cs);
        table[t * P + j] = make_float2(cs, p.sign * sn);
    }
    __syncthreads();
    const int tail = p.d - 2 * P, items = P + tail;
    const int heads = (p.H + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * heads, hn = min(heads, p.H - h0);
    const int both = k ? 2 : 1;
    for (int i = threadIdx.x; i < both * hn * tn * items; i += THREADS) {
        const int it = i % items;
        int rest = i / items;
        const int t = rest % tn;
        rest /= tn;
        const int h = h0 + rest % hn;
        const bool is_k = rest / hn > 0;
        const View vi = is_k ? p.ki : p.qi, vo = is_k ? p.ko : p.qo;
        const T* src = (is_k ? k : q) + b * vi.b + h * vi.h + (t0 + t) * vi.n;
        T* dst = (is_k ? kout : qout) + b * vo.b + h * vo.h + (t0 + t) * vo.n;
        if (it >= P) {
            dst[P + it] = src[P + it];
            continue;
        }
        int e1 = 2 * it, e2 = 2 * it + 1;
        if (!p.interleaved) {
            int a = 0;
            while (a + 1 < p.ax.n && 2 * it >= p.ax.at[a + 1]) ++a;
            e1 = p.ax.at[a] / 2 + it;
            e2 = e1 + p.ax.dims[a] / 2;
        }
        const float2 cs = table[t * P + it];
        const float x = to_f(src[e1]), y = to_f(src[e2]);
        dst[e1] = from_f<T>(x * cs.x - y * cs.y);
        dst[e2] = from_f<T>(y * cs.x + x * cs.y);
    }
}

}  // namespace rope

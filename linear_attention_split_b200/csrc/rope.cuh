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
// keeps the table in shared memory for its heads and both tensors.
//
// The floor is HBM (one read and one write of Q and K); what bounds it is the latency of the loads.  A thread takes VEC adjacent pairs: two
// loads of VEC features (16 bytes each where dims, strides and pointers are multiples of 16 bytes;
// the largest power of two that divides them all otherwise), two table reads, two stores.  A unit
// (its place in the head) is fixed for a thread; it walks rows, several loads in flight, and finds a row's head
// and token by shifts (TN is a power of two).  Two clips of 8 x 24 x 24 tokens, 12 heads of 128, bf16: 21.8 us,
// 5.2 TB/s (22.6 with a division per row, 24.8 with one per entry of the table as well; then blocks of 8 or 32
// tokens took 26.7 and 29.4, three or five blocks an SM 30 and 42).  Sections whose halves are odd go by
// single features: 1.5 TB/s.
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
    int H, N, TN;
    int heads;             // heads of a block
    int units, tail;       // units of a head: pairs / VEC turned, then tail / VEC passed on
    int interleaved;
    float sign;            // -1: inverse
    Axes ax;
    View qi, ki, qo, ko;
    double turns[MAX_D / 2];  // frequency of each pair / 2 pi
};

// VEC features as they lie in memory
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Lane {
    T v[VEC];
};

// The rotation, written so that every variant rounds alike (the compiler chooses no contraction)
__device__ __forceinline__ void turn(float x, float y, float c, float s, float& a, float& b) {
    a = fmaf(x, c, -__fmul_rn(y, s));
    b = fmaf(y, c, __fmul_rn(x, s));
}

template <typename T, int VEC>
__global__ void __launch_bounds__(THREADS, 4)
    rope_kernel(const T* q, const T* k, T* qout, T* kout, const __grid_constant__ Params p) {
    extern __shared__ __align__(16) float table[];  // [TN][pairs] cos, then the same of sin
    using L = Lane<T, VEC>;
    constexpr int FLY = sizeof(L) == 16 ? 2 : 4;  // rows of a thread that are in flight
    const int t0 = blockIdx.x * p.TN, tn = min(p.TN, p.N - t0);
    const int b = blockIdx.z, P = p.ax.pairs;
    float *cosines = table, *sines = table + p.TN * P;
    // launched with programmatic stream serialization: the table of a token grid depends on nothing the
    // previous grid wrote, so it overlaps that grid's tail
    if (p.pos) griddep_wait();
    // a thread keeps its pair (there are at most THREADS), its axis and frequency with it, and walks tokens
    static_assert(MAX_D / 2 <= THREADS, "a thread for each pair");
    const int apart = THREADS / P, j0 = threadIdx.x % P, first_t = threadIdx.x / P;
    if (first_t < apart) {
        int a = 0, inner = 1;  // cells of one step of the axis, on a token grid
        while (a + 1 < p.ax.n && 2 * j0 >= p.ax.at[a + 1]) ++a;
        for (int c = a + 1; c < p.ax.n; ++c) inner *= p.pos ? 1 : p.ax.grid[c];
        const double turns = p.turns[j0];
        for (int t = first_t; t < tn; t += apart) {
            const int tok = t0 + t;
            const double x = p.pos ? (double)p.pos[b * p.pos_b + (long long)tok * p.ax.n + a] : (double)(tok / inner % p.ax.grid[a]);
            double r = x * turns;
            r -= rint(r);
            float sn, cs;
            sincospif(2.f * (float)r, &sn, &cs);
            cosines[t * P + j0] = cs;
            sines[t * P + j0] = p.sign * sn;
        }
    }
    if (!p.pos) griddep_wait();
    griddep_launch();
    __syncthreads();
    // threads are laid out [rows at a time][units]; a row is (tensor, head, token)
    const int all = p.units + p.tail, rpp = max(1, THREADS / all);
    const int unit0 = threadIdx.x % all, r0 = threadIdx.x / all;
    if (r0 >= rpp && all <= THREADS) return;
    const int h0 = blockIdx.y * p.heads, hn = min(p.heads, p.H - h0);
    const int lg = 31 - __clz(p.TN), rows = (k ? 2 : 1) * hn << lg;  // a last tile's missing tokens count as rows
    for (int unit = unit0; unit < all; unit += THREADS) {  // more than one pass only for heads wider than the block
        int e1 = 2 * VEC * unit, e2 = e1 + VEC, j = VEC * unit;
        const bool turned = unit < p.units;
        if (!turned) {
            e1 = e2 = 2 * P + (unit - p.units) * VEC;
        } else if (!p.interleaved) {
            int a = 0;
            while (a + 1 < p.ax.n && 2 * j >= p.ax.at[a + 1]) ++a;
            e1 = p.ax.at[a] / 2 + j;
            e2 = e1 + p.ax.dims[a] / 2;
        }
        for (int first = r0; first < rows; first += FLY * rpp) {
            L x[FLY], y[FLY];
            T* dst[FLY];
            int tok[FLY];
#pragma unroll
            for (int f = 0; f < FLY; ++f) {
                const int row = first + f * rpp;
                const int hh = row >> lg, t = row - (hh << lg);
                tok[f] = row < rows && t < tn ? t : -1;
                if (tok[f] < 0) continue;
                const bool is_k = hh >= hn;
                const int h = h0 + (is_k ? hh - hn : hh);
                const View& vi = is_k ? p.ki : p.qi;
                const View& vo = is_k ? p.ko : p.qo;
                const T* src = (is_k ? k : q) + b * vi.b + h * vi.h + (t0 + t) * vi.n;
                dst[f] = (is_k ? kout : qout) + b * vo.b + h * vo.h + (t0 + t) * vo.n;
                x[f] = *reinterpret_cast<const L*>(src + e1);
                if (turned) y[f] = *reinterpret_cast<const L*>(src + e2);
            }
#pragma unroll
            for (int f = 0; f < FLY; ++f) {
                if (tok[f] < 0) continue;
                if (!turned) {
                    *reinterpret_cast<L*>(dst[f] + e1) = x[f];
                    continue;
                }
                const float *cp = cosines + tok[f] * P + j, *sp = sines + tok[f] * P + j;
                float c[VEC], s[VEC];
                if constexpr (VEC >= 4) {
#pragma unroll
                    for (int e = 0; e < VEC; e += 4) {
                        const float4 cv = *reinterpret_cast<const float4*>(cp + e), sv = *reinterpret_cast<const float4*>(sp + e);
                        c[e] = cv.x, c[e + 1] = cv.y, c[e + 2] = cv.z, c[e + 3] = cv.w;
                        s[e] = sv.x, s[e + 1] = sv.y, s[e + 2] = sv.z, s[e + 3] = sv.w;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) c[e] = cp[e], s[e] = sp[e];
                }
                L o1, o2;
                if (p.interleaved) {  // pairs are neighbours: VEC pairs in the 2 VEC features of x, y
                    float in[2 * VEC], out[2 * VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) in[e] = to_f(x[f].v[e]), in[VEC + e] = to_f(y[f].v[e]);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        turn(in[2 * e], in[2 * e + 1], c[e], s[e], out[2 * e], out[2 * e + 1]);
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o1.v[e] = from_f<T>(out[e]), o2.v[e] = from_f<T>(out[VEC + e]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        float a, d;
                        turn(to_f(x[f].v[e]), to_f(y[f].v[e]), c[e], s[e], a, d);
                        o1.v[e] = from_f<T>(a);
                        o2.v[e] = from_f<T>(d);
                    }
                }
                *reinterpret_cast<L*>(dst[f] + e1) = o1;
                *reinterpret_cast<L*>(dst[f] + e2) = o2;
            }
        }
    }
}

}  // namespace rope

// Linear cross attention to an encoder's tokens, forward, backward and for single
// tokens (la_forward_cross, la_backward_cross, la_decode_step_cross in
// include/linattn.h).  With f = phi(q_i), g = phi(k_j):
//   S = sum_j g_j v_j^T,  z = sum_j g_j,  y_i = S^T f_i / den_i,  den_i = f_i . z;
// backwards, with r_i = 1 / den_i,
//   G_i = S dy_i,  t_i = r_i f_i . G_i (which is y_i . dy_i),
//   df_i = r_i (G_i - t_i z),
//   dS = sum_i r_i f_i dy_i^T,  dz = -sum_i r_i t_i f_i,
//   dg_j = dS v_j + dz,  dv_j = dS^T g_j,
// and dq, dk are df, dg times phi'.  Neither the outputs nor anything else of a
// token's is kept from the forward: S and z are all that the backward needs.
//
// This file has the argument checks, the fp32 kernels on CUDA cores, which take any head
// size and stride and reach a third of what the fp32 units could (23 to 25 TFLOP/s on 8 x 8
// x 2048 to 2048 x 128), and the single tokens' kernel.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "la_cross.h"
#include "la_internal.h"
#include "la_layer.cuh"
#include "la_tc.h"
#include "la_tc_host.h"
#include "la_tc_ptx.cuh"

namespace la {
namespace cross {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float phi_of(float x, int phi) {
    if (!phi) return x;
    const float e = expf(fminf(x, 0.f));
    return x > 0.f ? x + 1.f : x <= 0.f ? e : x;  // NaN of NaN
}
__device__ __forceinline__ float slope_of(float x, int phi) {
    return !phi || x > 0.f ? 1.f : expf(x);
}

// ---------------------------------------------------------------- sums of outer products

// Number i of a thread's M of a tile's side, from its place t in 16: runs of four, 64
// apart, so that a warp's 16-byte reads of shared memory meet no bank twice.
__device__ __forceinline__ int in_tile(int t, int i) { return i / 4 * 64 + t * 4 + i % 4; }

template <int M>
__device__ __forceinline__ void read_side(const float *row, int t, float (&v)[M]) {
#pragma unroll
    for (int i = 0; i < M; i += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(row + in_tile(t, i));
        v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
    }
}

// S[a][c] += w_i f(x_i)[a] y_i[c] and z[a] += u_i w_i f(x_i)[a] over a part of the
// tokens, w = r or 1 and u = -t or 1: kTile x kTile sums per block, M x M per thread.
template <int kTile>
__global__ void __launch_bounds__(kThreads, 2) sum_kernel(const SumParams p) {
    constexpr int kTok = 16, kPitch = kTile + 4, M = kTile / 16;
    __shared__ __align__(16) float A[kTok][kPitch], Y[kTok][kPitch];
    __shared__ float U[kTok];
    const int tiles = (p.d + kTile - 1) / kTile;
    const long long head = blockIdx.x / (tiles * tiles);
    const int tile = (int)(blockIdx.x - head * (tiles * tiles)), seg = blockIdx.y;
    const int a0 = tile / tiles * kTile, c0 = tile % tiles * kTile;
    const int b = (int)(head / p.Hk), h = (int)(head % p.Hk);
    const int len = tokens_of(p.lengths, b, p.L);
    const long long all = (long long)p.group * p.L;
    const long long i0 = seg * p.per, i1 = min(i0 + p.per, all);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[M][M] = {}, zacc[M] = {};
    // a thread brings feature f of some rows, the next tokens' while these are summed
    constexpr int kPer = kTok * kTile / kThreads, kStep = kThreads / kTile;
    const int f = threadIdx.x % kTile, r0 = threadIdx.x / kTile;
    const bool in_x = a0 + f < p.d, in_y = c0 + f < p.d;
    const float *xs = static_cast<const float *>(p.x) + b * p.sx.b + a0 + f;
    const float *ys = static_cast<const float *>(p.y) + b * p.sy.b + c0 + f;
    float x[kPer], y[kPer];
    float2 rt[kPer];
    int g0 = (int)(i0 / max(p.L, 1)), n0 = (int)(i0 - (long long)g0 * p.L);  // of token i
    auto fetch = [&](long long i) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int row = r0 + k * kStep;
            int g = g0, n = n0 + row;
            if (n >= p.L) g += n / p.L, n %= p.L;
            const bool ok = i + row < i1 && n < len;
            const long long hh = (long long)h * p.group + g;
            x[k] = y[k] = 0.f;
            rt[k] = make_float2(ok ? 1.f : 0.f, -1.f);
            if (ok && p.rt) rt[k] = p.rt[(head * p.group + g) * p.L + n];
            if (ok && in_x) x[k] = xs[hh * p.sx.h + n * p.sx.n];
            if (ok && in_y) y[k] = ys[hh * p.sy.h + n * p.sy.n];
        }
        n0 += kTok;
        if (n0 >= p.L) g0 += n0 / p.L, n0 %= p.L;
    };
    const long long end = p.group == 1 ? min(i1, (long long)len) : i1;
    if (i0 < end) fetch(i0);
    for (long long i = i0; i < end; i += kTok) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int row = r0 + k * kStep;
            const bool none = is_none(rt[k]);
            A[row][f] = in_x ? rt[k].x * phi_of(x[k], p.phi) : 0.f;
            Y[row][f] = none ? 0.f : y[k];
            if (f == 0) U[row] = none ? 0.f : -rt[k].y;
        }
        __syncthreads();
        if (i + kTok < end) fetch(i + kTok);
#pragma unroll
        for (int row = 0; row < kTok; ++row) {
            float av[M], yv[M];
            read_side(A[row], ty, av);
            read_side(Y[row], tx, yv);
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int n = 0; n < M; ++n) acc[m][n] = fmaf(av[m], yv[n], acc[m][n]);
            if (tx == 0)
#pragma unroll
                for (int m = 0; m < M; ++m) zacc[m] = fmaf(av[m], U[row], zacc[m]);
        }
    }
    float *S = p.S + (seg * p.heads + head) * p.d * p.d;
    float *z = p.z + (seg * p.heads + head) * p.d;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int a = a0 + in_tile(ty, m);
        if (a >= p.d) continue;
#pragma unroll
        for (int n = 0; n < M; ++n) {
            const int c = c0 + in_tile(tx, n);
            if (c < p.d) S[a * p.d + c] = acc[m][n];
        }
        if (tx == 0 && c0 == 0) z[a] = zacc[m];
    }
}

// The parts of the states together, in order: out[i] = sum over segs of part[seg][i].
__global__ void __launch_bounds__(kThreads)
join_kernel(const float *S_part, const float *z_part, float *S, float *z, long long nS,
            long long nz, int segs) {
    for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < nS + nz;
         i += (long long)gridDim.x * kThreads) {
        const bool inS = i < nS;
        const float *from = inS ? S_part + i : z_part + (i - nS);
        const long long step = inS ? nS : nz;
        float t[4] = {};
        int s = 0;
        for (; s + 4 <= segs; s += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] += from[(s + e) * step];
        for (; s < segs; ++s) t[0] += from[s * step];
        (inS ? S[i] : z[i - nS]) = (t[0] + t[1]) + (t[2] + t[3]);
    }
}

// ---------------------------------------------------------------- rows times a state

// y_i = S^T f(x_i), over f . z with norm: kTile rows x kTile columns per block, M x M
// per thread.  (8 x 8 x 2048 x 128: 164 us with all the registers a thread takes, 191 us
// with half of them.)
template <int kTile>
__global__ void __launch_bounds__(kThreads, 1) read_kernel(const ReadParams p) {
    constexpr int kStep = 16, kPitch = kTile + 4, M = kTile / 16;
    __shared__ __align__(16) float A[kStep][kPitch], Y[kStep][kPitch];
    __shared__ float Z[kStep];
    const int tiles = (p.d + kTile - 1) / kTile, row_tiles = (p.L + kTile - 1) / kTile;
    const long long u = blockIdx.x / tiles;
    const int c0 = (int)(blockIdx.x - u * tiles) * kTile;
    const long long bh = u / row_tiles;  // of x's heads
    const int n0 = (int)(u - bh * row_tiles) * kTile;
    const int H = p.Hk * p.group, b = (int)(bh / H), h = (int)(bh % H);
    const long long state = (long long)b * p.Hk + h / p.group;
    const int len = tokens_of(p.lengths, b, p.L);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float *x = static_cast<const float *>(p.x) + b * p.sx.b + h * p.sx.h;
    const float *S = p.S + state * p.d * p.d;
    float acc[M][M] = {}, den[M] = {};
    // the next features' values come while these are multiplied
    constexpr int kPer = kTile * kStep / kThreads;
    float av[kPer], yv[kPer], zv = 0.f;
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x + i * kThreads;
            const int row = n0 + e / kStep, f = k0 + e % kStep, a = k0 + e / kTile,
                      c = c0 + e % kTile;
            av[i] = row < len && f < p.d ? x[row * p.sx.n + f] : 0.f;
            yv[i] = a < p.d && c < p.d ? S[a * p.d + c] : 0.f;
        }
        if (threadIdx.x < kStep)
            zv = p.norm && k0 + (int)threadIdx.x < p.d ? p.z[state * p.d + k0 + threadIdx.x] : 0.f;
    };
    fetch(0);
    for (int k0 = 0; k0 < p.d; k0 += kStep) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x + i * kThreads;
            // features from d on meet zeros of S; rows behind the length are not used
            A[e % kStep][e / kStep] = phi_of(av[i], p.phi);
            Y[e / kTile][e % kTile] = yv[i];
        }
        if (threadIdx.x < kStep) Z[threadIdx.x] = zv;
        __syncthreads();
        if (k0 + kStep < p.d) fetch(k0 + kStep);
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            float a[M], y[M];
            read_side(A[k], ty, a);
            read_side(Y[k], tx, y);
            const float z = Z[k];
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int n = 0; n < M; ++n) acc[m][n] = fmaf(a[m], y[n], acc[m][n]);
                den[m] = fmaf(a[m], z, den[m]);
            }
        }
    }
    float *y = static_cast<float *>(p.y) + b * p.sy.b + h * p.sy.h;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int n = n0 + in_tile(ty, m);
        if (n >= p.L) continue;
#pragma unroll
        for (int e = 0; e < M; ++e) {
            const int c = c0 + in_tile(tx, e);
            if (c >= p.d) continue;
            // without keys there is nothing to average: 0
            const float v = !p.norm ? acc[m][e] : den[m] == 0.f ? 0.f : acc[m][e] / den[m];
            y[n * p.sy.n + c] = n < len ? v : 0.f;
        }
    }
}

// G_i = S y_i, and from it the gradient of row i: on q's side
// r (G - t z) phi'(x) with r and t left for the sums, on k's side (G + z) phi'(x)
// (z is then dz).  A warp takes 4 rows whole, a lane every 32nd feature.
template <int kCols>  // kCols: 32 features each, of d
__global__ void __launch_bounds__(kThreads) grad_kernel(const GradParams p) {
    constexpr int kRows = 32, kStep = 32, kPerY = kRows * kStep / kThreads;
    constexpr int kPerW = kCols * 32 * kStep / kThreads;
    __shared__ float Y[kRows][kStep], W[kCols * 32][kStep + 1];
    const int row_tiles = (p.L + kRows - 1) / kRows;
    const long long bh = blockIdx.x / row_tiles;
    const int n0 = (int)(blockIdx.x - bh * row_tiles) * kRows;
    const int H = p.Hk * p.group, b = (int)(bh / H), h = (int)(bh % H);
    const long long state = (long long)b * p.Hk + h / p.group;
    const int len = tokens_of(p.lengths, b, p.L);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float *y = static_cast<const float *>(p.y) + b * p.sy.b + h * p.sy.h;
    const float *x = static_cast<const float *>(p.x) + b * p.sx.b + h * p.sx.h;
    // the next features' values come while these are multiplied
    float yv[kPerY], wv[kPerW];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kPerY; ++i) {
            const int e = threadIdx.x + i * kThreads, row = e / kStep, c = e % kStep;
            yv[i] = n0 + row < len && k0 + c < p.d ? y[(n0 + row) * p.sy.n + k0 + c] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kPerW; ++i) {
            const int e = threadIdx.x + i * kThreads, a = e / kStep, c = e % kStep;
            wv[i] = a < p.d && k0 + c < p.d ? p.S[(state * p.d + a) * p.d + k0 + c] : 0.f;
        }
    };
    fetch(0);
    float acc[4][kCols] = {};
    for (int k0 = 0; k0 < p.d; k0 += kStep) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPerY; ++i) {
            const int e = threadIdx.x + i * kThreads;
            Y[e / kStep][e % kStep] = yv[i];
        }
#pragma unroll
        for (int i = 0; i < kPerW; ++i) {
            const int e = threadIdx.x + i * kThreads;
            W[e / kStep][e % kStep] = wv[i];
        }
        __syncthreads();
        if (k0 + kStep < p.d) fetch(k0 + kStep);
#pragma unroll 4
        for (int k = 0; k < kStep; ++k) {
            float v[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) v[m] = Y[warp * 4 + m][k];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const float w = W[lane + 32 * j][k];
#pragma unroll
                for (int m = 0; m < 4; ++m) acc[m][j] = fmaf(w, v[m], acc[m][j]);
            }
        }
    }
    float *dx = static_cast<float *>(p.dx) + b * p.sdx.b + h * p.sdx.h;
    float xv[4][kCols], zv[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        const int a = lane + 32 * j;
        zv[j] = a < p.d && (p.norm || p.keys) ? p.z[state * p.d + a] : 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int n = n0 + warp * 4 + m;
            xv[m][j] = a < p.d && n < len ? x[n * p.sx.n + a] : 0.f;
        }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int n = n0 + warp * 4 + m;
        if (n >= p.L) continue;
        float dot = 0.f, den = 0.f;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (lane + 32 * j < p.d) {
                const float f = phi_of(xv[m][j], p.phi);
                dot = fmaf(f, acc[m][j], dot);
                den = fmaf(f, zv[j], den);
            }
        float r = 1.f, t = p.keys ? -1.f : 0.f;
        bool none = false;
        if (!p.keys) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                dot += __shfl_xor_sync(~0u, dot, o);
                den += __shfl_xor_sync(~0u, den, o);
            }
            if (p.norm) {
                none = den == 0.f;
                r = none ? 0.f : 1.f / den;
                t = dot * r;
            }
            if (lane == 0) p.rt[bh * p.L + n] = none ? no_row() : make_float2(r, t);
        }
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const int a = lane + 32 * j;
            if (a >= p.d) continue;
            const float g = r * fmaf(-t, zv[j], acc[m][j]) * slope_of(xv[m][j], p.phi);
            dx[n * p.sdx.n + a] = n < len && !none ? g : 0.f;
        }
    }
}

// ---------------------------------------------------------------- single tokens

struct StepParams {
    const float *S, *z;
    const void *q;
    void *out;
    la_strides sq, so;
    int Hk, G, N, d, phi, norm;
};

// kR queries of one state: the state is read once, a row of it by as many threads as
// it has vectors of V, the rows in turn by the rest.  Bound by that read: 256 x 32 states
// of 128 x 128 in 91 us, 6.0 TB/s.  (Vectors of 32 bytes 97 us; 16 rows under way per
// thread instead of 8 94 us.)
template <typename T, int kR, int V>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepParams p) {
    __shared__ float F[kR][LA_MAX_D], den[kR];
    __shared__ __align__(16) float sum[kThreads * V];
    const int rows = p.G * p.N, chunks = (rows + kR - 1) / kR;
    const long long state = blockIdx.x / chunks;
    const int r0 = (int)(blockIdx.x - state * chunks) * kR;
    const int b = (int)(state / p.Hk), h = (int)(state % p.Hk);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto offset = [&](const la_strides &s, int r) {
        const int g = r / p.N, n = r - g * p.N;
        return b * s.b + (long long)(h * p.G + g) * s.h + n * s.n;
    };
    const int vecs = (p.d + V - 1) / V;
    int lanes = 1;
    while (lanes < vecs) lanes <<= 1;
    const int c = threadIdx.x & (lanes - 1), part = threadIdx.x / lanes;
    const int parts = kThreads / lanes;

    for (int i = threadIdx.x; i < kR * p.d; i += kThreads) {
        const int r = i / p.d, a = i - r * p.d;
        F[r][a] = r0 + r < rows
                      ? phi_of(to_f(static_cast<const T *>(p.q)[offset(p.sq, r0 + r) + a]), p.phi)
                      : 0.f;
    }
    __syncthreads();
    if (p.norm)
        for (int r = warp; r < kR; r += kThreads / 32) {
            float t = 0.f;
            for (int a = lane; a < p.d; a += 32) t = fmaf(F[r][a], p.z[state * p.d + a], t);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
            if (lane == 0) den[r] = t;
        }
    float acc[kR][V] = {};
    if (c < vecs) {
        const float *S = p.S + state * p.d * p.d + c * V;
#pragma unroll 8
        for (int a = part; a < p.d; a += parts) {
            const Pack<float, V> w = *reinterpret_cast<const Pack<float, V> *>(S + a * p.d);
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int e = 0; e < V; ++e) acc[r][e] = fmaf(F[r][a], w.v[e], acc[r][e]);
        }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) sum[threadIdx.x * V + e] = acc[r][e];
        __syncthreads();
        if (r0 + r < rows && threadIdx.x < p.d) {
            float t = 0.f;
            for (int q = 0; q < parts; ++q) t += sum[q * lanes * V + threadIdx.x];
            if (p.norm) t = den[r] == 0.f ? 0.f : t / den[r];
            from_f(static_cast<T *>(p.out)[offset(p.so, r0 + r) + threadIdx.x], t);
        }
    }
}

// ---------------------------------------------------------------- launches

cudaError_t counted(cudaError_t e) {
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) note_launches(1);
    return e;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The side of the fp32 sums' square tiles: 8 x 8 values per thread, which read the least
// of shared memory, where a tile of 128 is not mostly empty and there are enough of them
// (8 x 8 x 2048 x 128 into states: 175 us, 465 us by 4 x 4; forward of 16 heads x
// 1024 x 96 52 us, 60 us with 64; of 8 heads x 512 x 128 31 us, 23 us with 64).
int tile_of(const Shape &sh, long long tokens, int sms) {
    const long long side = (sh.d + 127) / 128;
    return sh.d > 64 && sh.heads() * side * side * (tokens / 256) >= sms / 3 ? 128 : 64;
}

// Parts of the tokens of one head's sums: enough that all SMs are busy three times over,
// and of at most 1024 tokens each (a longer chain of fp32 additions rounds more off) as
// long as the parts of all states stay within 256 MB.
Cut cut_of(const Shape &sh, la_dtype dtype, long long tokens, int sms) {
    Cut c;
    c.tile = tile_of(sh, tokens, sms);
    const int side = (sh.d + c.tile - 1) / c.tile;
    const int tiles = dtype == LA_F32 ? side * side : (sh.d + 63) / 64;  // of a state
    const long long blocks = std::max(1LL, sh.heads() * tiles);
    const long long most = (1LL << 26) / std::max(1LL, sh.heads() * (sh.state() + sh.d));
    long long segs = std::max(std::min((tokens + 1023) / 1024, most),
                              std::min((3LL * sms + blocks - 1) / blocks, tokens / 64));
    segs = std::max(1LL, std::min(segs, 65535LL));
    c.per = ((tokens + segs - 1) / segs + 15) / 16 * 16;
    c.segs = c.per ? (int)((tokens + c.per - 1) / c.per) : 1;
    if (c.segs < 1) c.segs = 1;
    return c;
}

size_t part_bytes(const Shape &sh, const Cut &c) {
    return c.segs == 1 ? 0
                       : up(sizeof(float) * (size_t)c.segs * sh.heads() * sh.state()) +
                             up(sizeof(float) * (size_t)c.segs * sh.heads() * sh.d);
}

struct Plan {
    Cut keys, queries;
    size_t off_dS, off_dz, off_rt, off_part, total;
};

// The workspace serves either set of kernels: the tensors' strides decide which runs.
Plan plan_of(const Shape &sh, la_dtype dtype, int sms, bool back) {
    Plan p{};
    const size_t tc = dtype == LA_BF16 && sh.d <= 128 && sh.d % 8 == 0
                          ? tc_workspace(sh, sms, back) : 0;
    p.keys = cut_of(sh, dtype, sh.M, sms);
    p.queries = cut_of(sh, dtype, (long long)sh.G() * sh.N, sms);
    if (!back) {
        p.total = std::max(tc, part_bytes(sh, p.keys));
        return p;
    }
    p.off_dz = up(sizeof(float) * (size_t)sh.heads() * sh.state());
    p.off_rt = p.off_dz + up(sizeof(float) * (size_t)sh.heads() * sh.d);
    p.off_part = p.off_rt + up(sizeof(float2) * (size_t)sh.B * sh.Hq * sh.N);
    p.total = std::max(tc, p.off_part + part_bytes(sh, p.queries));
    return p;
}

// The sums over x's and y's tokens into S and z, through `part` where they are cut.
template <typename T>
cudaError_t sums(const Shape &sh, Rows x, Rows y, int group, int L, const float2 *rt,
                 const int *lengths, Cut cut, float *S, float *z, char *part, cudaStream_t s) {
    SumParams p{};
    p.x = x.x;
    p.y = y.x;
    p.sx = x.s;
    p.sy = y.s;
    p.rt = rt;
    p.lengths = lengths;
    p.Hk = sh.Hk;
    p.group = group;
    p.L = L;
    p.d = sh.d;
    p.phi = sh.phi;
    p.segs = cut.segs;
    p.per = cut.per;
    p.heads = sh.heads();
    float *pz = reinterpret_cast<float *>(
        part + up(sizeof(float) * (size_t)cut.segs * sh.heads() * sh.state()));
    p.S = cut.segs == 1 ? S : reinterpret_cast<float *>(part);
    p.z = cut.segs == 1 ? z : pz;
    cudaError_t e = cudaSuccess;
    if constexpr (sizeof(T) == 2) {
        e = half_sums(p, s);
    } else {
        const int tiles = (sh.d + cut.tile - 1) / cut.tile;
        const dim3 grid((unsigned)(sh.heads() * tiles * tiles), (unsigned)cut.segs);
        if (cut.tile == 128)
            sum_kernel<128><<<grid, kThreads, 0, s>>>(p);
        else
            sum_kernel<64><<<grid, kThreads, 0, s>>>(p);
        e = counted(cudaSuccess);
    }
    if (e != cudaSuccess || cut.segs == 1) return e;
    const long long nS = sh.heads() * sh.state(), nz = sh.heads() * sh.d;
    const unsigned blocks = (unsigned)std::min((nS + nz + kThreads - 1) / kThreads, 4096LL);
    join_kernel<<<blocks, kThreads, 0, s>>>(p.S, p.z, S, z, nS, nz, cut.segs);
    return counted(cudaSuccess);
}

template <typename T>
cudaError_t read(const Shape &sh, Rows x, Rows y, int group, int L, const float *S,
                 const float *z, int norm, const int *lengths, cudaStream_t s) {
    ReadParams p{x.x, y.x, x.s, y.s, S, z, lengths, sh.Hk, group, L, sh.d, sh.phi, norm};
    // Tiles of 64 where those of 128 would be half empty (8192 states, 32 rows of each: 650
    // us, 980 us with 128) or leave SMs without one (4 x 256 rows, 256 keys: forward 30 us, 42
    // us with 128; 2 x 16 x 1024 rows: 111 us, 102 us with 128).
    const long long heads = sh.heads() * group;
    if (heads == 0) return cudaSuccess;
    if constexpr (sizeof(T) == 2) return half_read(p, heads, s);
    int sms = 0;
    const cudaError_t e = tchost::sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int tile = sh.d > 64 && L > 64 && heads * ((L + 127) / 128) * ((sh.d + 127) / 128) >= sms ? 128 : 64;
    const long long blocks =
        heads * (((long long)L + tile - 1) / tile) * ((sh.d + tile - 1) / tile);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (tile == 128)
        read_kernel<128><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    else
        read_kernel<64><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return counted(cudaSuccess);
}

template <typename T>
cudaError_t grads(const Shape &sh, Rows y, Rows x, Rows dx, int group, int L, const float *S,
                  const float *z, float2 *rt, const int *lengths, int keys, cudaStream_t s) {
    GradParams p{y.x, x.x, dx.x, y.s, x.s, dx.s, S, z, rt, lengths,
                 sh.Hk, group, L, sh.d, sh.phi, sh.norm, keys};
    if (sh.heads() * group == 0) return cudaSuccess;
    if constexpr (sizeof(T) == 2) return half_grads(p, sh.heads() * group, s);
    const long long blocks = sh.heads() * group * ((L + 31) / 32);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    auto go = [&](auto kern) {
        kern<<<(unsigned)blocks, kThreads, 0, s>>>(p);
        return counted(cudaSuccess);
    };
    if (sh.d <= 32) return go(grad_kernel<1>);
    if (sh.d <= 64) return go(grad_kernel<2>);
    if (sh.d <= 96) return go(grad_kernel<3>);
    if (sh.d <= 128) return go(grad_kernel<4>);
    return go(grad_kernel<8>);
}

template <typename T>
cudaError_t forward(const Shape &sh, const Plan &pl, Rows q, Rows k, Rows v, Rows out, float *S,
                    float *z, char *ws, cudaStream_t s) {
    cudaError_t e =
        sums<T>(sh, k, v, 1, sh.M, nullptr, sh.lengths, pl.keys, S, z, ws, s);
    if (e != cudaSuccess || sh.N == 0) return e;
    return read<T>(sh, q, out, sh.G(), sh.N, S, z, sh.norm, nullptr, s);
}

template <typename T>
cudaError_t backward(const Shape &sh, const Plan &pl, Rows dout, Rows q, Rows k, Rows v,
                     const float *S, const float *z, Rows dq, Rows dk, Rows dv, char *ws,
                     cudaStream_t s) {
    float *dS = reinterpret_cast<float *>(ws), *dz = reinterpret_cast<float *>(ws + pl.off_dz);
    float2 *rt = reinterpret_cast<float2 *>(ws + pl.off_rt);
    cudaError_t e = cudaSuccess;
    if (sh.N > 0)
        e = grads<T>(sh, dout, q, dq, sh.G(), sh.N, S, z, rt, nullptr, 0, s);
    if (e != cudaSuccess || sh.M == 0) return e;
    e = sums<T>(sh, q, dout, sh.G(), sh.N, rt, nullptr, pl.queries, dS, dz, ws + pl.off_part, s);
    if (e == cudaSuccess)
        e = grads<T>(sh, v, k, dk, 1, sh.M, dS, dz, nullptr, sh.lengths, 1, s);
    if (e == cudaSuccess) e = read<T>(sh, k, dv, 1, sh.M, dS, dz, 0, sh.lengths, s);
    return e;
}

template <typename T, int V>
cudaError_t launch_step(const StepParams &p, long long states, cudaStream_t s) {
    const long long rows = (long long)p.G * p.N;
    auto go = [&](auto kern, int per) {
        const long long blocks = states * ((rows + per - 1) / per);
        if (blocks > 0x7fffffff || rows > 0x7fffffff - 8) return cudaErrorInvalidConfiguration;
        kern<<<(unsigned)blocks, kThreads, 0, s>>>(p);
        return counted(cudaSuccess);
    };
    if (rows <= 1) return go(step_kernel<T, 1, V>, 1);
    if (rows <= 2) return go(step_kernel<T, 2, V>, 2);
    if (rows <= 4) return go(step_kernel<T, 4, V>, 4);
    return go(step_kernel<T, 8, V>, 8);
}

template <typename T>
cudaError_t step(const Shape &sh, Rows q, Rows out, const float *S, const float *z,
                 cudaStream_t s) {
    // Many tokens go as tiles, each of one head of queries; heads that share a state do not
    // make a tile fuller.  With 256 x 32 states of 128, 4 tokens take 154 us singly and 187 us
    // as a tile of la_cross_tc.cu, 8 take 231 and 188 (and 8 heads of one token, with 256 x 8
    // states, 65 and 179); with 128 x 16 of 100 in bf16 8 take 50 and 52, 12 take 98 and 54; in
    // fp32, 256 x 32 of 128, 16 take 437 and 641, 32 take 837 and 650.
    const Rows rows[2] = {q, out};
    if (sizeof(T) == 2 && sh.N > 4 && tc_rows(sh, rows, 2, nullptr, 0, S, z)) {
        int sms = 0;
        cudaError_t e = tchost::sm_count(&sms);
        int *status = e == cudaSuccess ? device_status_word(&e) : nullptr;
        return e == cudaSuccess ? tc_read(sh, q, out, S, z, false, sms, status, s) : e;
    }
    if (sh.N > (sizeof(T) == 2 ? 8 : 24))
        return read<T>(sh, q, out, sh.G(), sh.N, S, z, sh.norm, nullptr, s);
    const StepParams p{S, z, q.x, out.x, q.s, out.s, sh.Hk, sh.G(), sh.N, sh.d, sh.phi, sh.norm};
    return sh.d % 4 == 0 && (uintptr_t)S % 16 == 0 ? launch_step<T, 4>(p, sh.heads(), s)
                                                  : launch_step<T, 1>(p, sh.heads(), s);
}

// ---------------------------------------------------------------- checks

la_status shape_of(const char *who, Shape &sh, const int *lengths, int B, int Hq, int Hk, int N,
                   int M, int d, const la_variant *variant, la_dtype dtype) {
    if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || M < 0)
        return layer_fail(LA_ERR_INVALID_ARG, who, "negative B, Hq, Hk, N or M");
    if (d < 1 || d > LA_MAX_D) return layer_fail(LA_ERR_INVALID_ARG, who, "d must be in 1..256");
    if (dtype != LA_F32 && dtype != LA_BF16)
        return layer_fail(LA_ERR_INVALID_ARG, who, "unknown dtype");
    if (Hk == 0 ? Hq != 0 : Hq % Hk != 0)
        return layer_fail(LA_ERR_INVALID_ARG, who, "Hq must be a multiple of Hk");
    if (variant && ((variant->feature_map != LA_PHI_ELU1 &&
                     variant->feature_map != LA_PHI_IDENTITY) ||
                    (variant->normalise != 0 && variant->normalise != 1)))
        return layer_fail(LA_ERR_INVALID_ARG, who, "unknown variant");
    if ((uintptr_t)lengths % 4) return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned lengths");
    // (the last tile's rows are counted in 32 bits, too, some of them behind the tokens)
    constexpr int kMostTokens = 0x7fffffff - 255;
    if ((double)B * std::max(Hq, Hk) * ((double)std::max(N, M) + 1) > 1e10 ||
        (double)B * Hk * 64 > 2147483647.0 || std::max(N, M) > kMostTokens)
        return layer_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
    sh = {B, Hq, Hk, N, M, d, !variant || variant->feature_map == LA_PHI_ELU1,
          variant ? variant->normalise : 1, lengths};
    return LA_OK;
}

// One of the call's tensors: [B][H][L][d] at its strides, `written` or read.
la_status rows_of(const char *who, Rows &r, const void *x, const la_strides *s, int H, int L,
                  const Shape &sh, la_dtype dtype, bool written) {
    r = {const_cast<void *>(x), s ? *s : contiguous(H, L, sh.d)};
    if (sh.B == 0 || H == 0 || L == 0) return LA_OK;
    if (!x) return layer_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
    if ((uintptr_t)x % (dtype == LA_F32 ? 4 : 2))
        return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
    if (negative(r.s)) return layer_fail(LA_ERR_INVALID_ARG, who, "negative stride");
    if (written && !rows_disjoint(r.s, sh.B, H, L, sh.d))
        return layer_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
    return LA_OK;
}

la_status states_fine(const char *who, const float *S, const float *z) {
    if (!S || !z) return layer_fail(LA_ERR_INVALID_ARG, who, "null state pointer");
    if ((uintptr_t)S % 4 || (uintptr_t)z % 4)
        return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned state pointer");
    return LA_OK;
}

// The caller's workspace, or one of the stream's (then in `own`).
la_status workspace_of(const char *who, void *workspace, size_t bytes, size_t need, char **ws,
                       void **own, cudaStream_t s) {
    *own = nullptr;
    *ws = static_cast<char *>(workspace);
    if (need == 0) return LA_OK;
    if (workspace) {
        if (bytes < need || (uintptr_t)workspace % 16)
            return layer_fail(LA_ERR_INVALID_ARG, who,
                              "workspace too small or not 16-byte aligned");
        return LA_OK;
    }
    if (tc_workspace_alloc(own, need, s) != cudaSuccess) {
        (void)cudaGetLastError();
        *own = nullptr;
        return layer_fail(LA_ERR_NO_MEMORY, who, "workspace allocation");
    }
    *ws = static_cast<char *>(*own);
    return LA_OK;
}

la_status finish(const char *who, cudaError_t e, void *own, cudaStream_t s) {
    if (own) {
        const cudaError_t ef = cudaFreeAsync(own, s);
        if (e == cudaSuccess) e = ef;
    }
    if (e == cudaSuccess) return LA_OK;
    return layer_fail(e == cudaErrorInvalidConfiguration ? LA_ERR_UNSUPPORTED : LA_ERR_CUDA, who,
                      cudaGetErrorString(e));
}

template <int kIn, int kOut>
bool aliased(const void *const (&in)[kIn], const void *const (&out)[kOut]) {
    for (int i = 0; i < kOut; ++i) {
        if (!out[i]) continue;
        for (const void *x : in)
            if (x == out[i]) return true;
        for (int j = 0; j < i; ++j)
            if (out[j] == out[i]) return true;
    }
    return false;
}

}  // namespace
}  // namespace cross
}  // namespace la

using namespace la;
using namespace la::cross;

extern "C" {

__attribute__((visibility("default")))
la_status la_forward_cross(const void *q, const void *k, const void *v, void *out, float *S,
                           float *z, const int *lengths, const la_strides *strides, int B, int Hq,
                           int Hk, int N, int M, int d, const la_variant *variant, la_dtype dtype,
                           void *workspace, size_t workspace_bytes, la_stream_t stream) {
    const char *who = "la_forward_cross";
    Shape sh;
    la_status st = shape_of(who, sh, lengths, B, Hq, Hk, N, M, d, variant, dtype);
    if (st != LA_OK) return st;
    if (B == 0 || Hk == 0) return LA_OK;
    Rows rq, rk, rv, ro;
    if ((st = rows_of(who, rq, q, strides, Hq, N, sh, dtype, false)) != LA_OK ||
        (st = rows_of(who, rk, k, strides ? strides + 1 : nullptr, Hk, M, sh, dtype, false)) !=
            LA_OK ||
        (st = rows_of(who, rv, v, strides ? strides + 2 : nullptr, Hk, M, sh, dtype, false)) !=
            LA_OK ||
        (st = rows_of(who, ro, out, strides ? strides + 3 : nullptr, Hq, N, sh, dtype, true)) !=
            LA_OK ||
        (st = states_fine(who, S, z)) != LA_OK)
        return st;
    if (aliased({q, k, v}, {static_cast<const void *>(out), S, z}))
        return layer_fail(LA_ERR_INVALID_ARG, who, "an output aliases another tensor");
    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e != cudaSuccess) return layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    const Plan pl = plan_of(sh, dtype, sms, false);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char *ws;
    void *own;
    st = workspace_of(who, workspace, workspace_bytes, pl.total, &ws, &own, s);
    if (st != LA_OK) return st;
    const Rows qs[2] = {rq, ro}, ks[2] = {rk, rv};
    if (dtype == LA_BF16 && M > 0 && tc_rows(sh, qs, N > 0 ? 2 : 0, ks, 2, S, z)) {
        int *status = device_status_word(&e);
        if (e == cudaSuccess) e = tc_state(sh, rk, rv, S, z, ws, sms, status, s);
        if (e == cudaSuccess && N > 0 && Hq > 0)
            e = tc_read(sh, rq, ro, S, z, true, sms, status, s);
    } else {
        e = dtype == LA_F32 ? forward<float>(sh, pl, rq, rk, rv, ro, S, z, ws, s)
                            : forward<__nv_bfloat16>(sh, pl, rq, rk, rv, ro, S, z, ws, s);
    }
    return finish(who, e, own, s);
}

__attribute__((visibility("default")))
la_status la_backward_cross(const void *dout, const void *q, const void *k, const void *v,
                            const float *S, const float *z, const int *lengths, void *dq,
                            void *dk, void *dv, const la_strides *strides, int B, int Hq, int Hk,
                            int N, int M, int d, const la_variant *variant, la_dtype dtype,
                            void *workspace, size_t workspace_bytes, la_stream_t stream) {
    const char *who = "la_backward_cross";
    Shape sh;
    la_status st = shape_of(who, sh, lengths, B, Hq, Hk, N, M, d, variant, dtype);
    if (st != LA_OK) return st;
    if (B == 0 || Hk == 0) return LA_OK;
    const void *x[7] = {dout, q, k, v, dq, dk, dv};
    Rows r[7];
    for (int i = 0; i < 7; ++i) {
        const bool queries = i < 2 || i == 4;
        st = rows_of(who, r[i], x[i], strides ? strides + i : nullptr, queries ? Hq : Hk,
                     queries ? N : M, sh, dtype, i >= 4);
        if (st != LA_OK) return st;
    }
    if ((st = states_fine(who, S, z)) != LA_OK) return st;
    if (aliased({dout, q, k, v, static_cast<const void *>(S), static_cast<const void *>(z)},
                {static_cast<const void *>(dq), static_cast<const void *>(dk),
                 static_cast<const void *>(dv)}))
        return layer_fail(LA_ERR_INVALID_ARG, who, "an output aliases another tensor");
    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e != cudaSuccess) return layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    const Plan pl = plan_of(sh, dtype, sms, true);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char *ws;
    void *own;
    st = workspace_of(who, workspace, workspace_bytes, pl.total, &ws, &own, s);
    if (st != LA_OK) return st;
    const Rows qs[3] = {r[0], r[1], r[4]}, ks[4] = {r[2], r[3], r[5], r[6]};
    if (dtype == LA_BF16 && M > 0 && N > 0 && Hq > 0 && tc_rows(sh, qs, 3, ks, 4, S, z)) {
        int *status = device_status_word(&e);
        if (e == cudaSuccess)
            e = tc_backward(sh, r[0], r[1], r[2], r[3], S, z, r[4], r[5], r[6], ws, sms, status, s);
        return finish(who, e, own, s);
    }
    e = dtype == LA_F32
            ? backward<float>(sh, pl, r[0], r[1], r[2], r[3], S, z, r[4], r[5], r[6], ws, s)
            : backward<__nv_bfloat16>(sh, pl, r[0], r[1], r[2], r[3], S, z, r[4], r[5], r[6], ws,
                                      s);
    return finish(who, e, own, s);
}

__attribute__((visibility("default")))
la_status la_decode_step_cross(const float *S, const float *z, const void *q, void *out,
                               const la_strides *strides, int B, int Hq, int Hk, int N, int d,
                               const la_variant *variant, la_dtype dtype, la_stream_t stream) {
    const char *who = "la_decode_step_cross";
    Shape sh;
    la_status st = shape_of(who, sh, nullptr, B, Hq, Hk, N, 0, d, variant, dtype);
    if (st != LA_OK) return st;
    if (B == 0 || Hq == 0 || N == 0) return LA_OK;
    Rows rq, ro;
    if ((st = rows_of(who, rq, q, strides, Hq, N, sh, dtype, false)) != LA_OK ||
        (st = rows_of(who, ro, out, strides ? strides + 1 : nullptr, Hq, N, sh, dtype, true)) !=
            LA_OK ||
        (st = states_fine(who, S, z)) != LA_OK)
        return st;
    if (aliased({q, static_cast<const void *>(S), static_cast<const void *>(z)},
                {static_cast<const void *>(out)}))
        return layer_fail(LA_ERR_INVALID_ARG, who, "out aliases an input");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return finish(who,
                  dtype == LA_F32 ? step<float>(sh, rq, ro, S, z, s)
                                  : step<__nv_bfloat16>(sh, rq, ro, S, z, s),
                  nullptr, s);
}

__attribute__((visibility("default")))
size_t la_cross_workspace_bytes(int B, int Hq, int Hk, int N, int M, int d, la_dtype dtype,
                                int backward) {
    if (B < 1 || Hk < 1 || Hq < 0 || Hq % Hk || N < 0 || M < 0 || d < 1 || d > LA_MAX_D) return 0;
    if (dtype != LA_F32 && dtype != LA_BF16) return 0;
    int sms = 0;
    if (tchost::sm_count(&sms) != cudaSuccess || sms <= 0) sms = 1;
    const Shape sh{B, Hq, Hk, N, M, d, 1, 1, nullptr};
    return plan_of(sh, dtype, sms, backward != 0).total;
}

}  // extern "C"

// Linear cross attention in bf16 for what the tiles of la_cross_tc.cu do not take (head
// sizes above 128 or not a multiple of 8, rows on other than 16-byte boundaries); the
// formulas are in la_cross.cu.
//
// The products are m16n8k16 of bf16 with fp32 sums, whose operands are staged in shared
// memory by plain loads of 8 bytes, or 2 where rows are not aligned.  Blocks cover all
// columns (kC: 64, 128 or 256), so that phi is taken of each value once, or once per 64
// features of the state (half_sum_kernel).
//
// What is rounded to bf16: phi(x) r as two numbers, high and low, for the sums, which are
// fp32 results (and end after 256 tokens, since the tensor cores cut off what they add);
// phi(x) and S as one each for the outputs and dv; S and dS as two for G = S dy and dS v,
// where large parts cancel.
//
// 8 x 8 (on 4) x 2048 to 2048 x 256: 190 us forward, 533 us backward (1367 and 2862 us by
// fp32 products on CUDA cores; on odd strides 278 and 766 us); 8 x 8 x 2048 to 2048 x 128 on
// odd strides 153 and 333 us (551 and 932).  Bound by instructions and latency, 0.3 to 0.5
// issued per cycle: addresses, phi and conversions on the way to shared memory, and the
// gradients' ends.
#include <cuda_bf16.h>

#include <algorithm>

#include "la_cross.h"
#include "la_internal.h"
#include "la_tc_ptx.cuh"

namespace la {
namespace cross {
namespace {

using T = __nv_bfloat16;

__device__ __forceinline__ float phi_fast(float x, int phi) {
    if (!phi) return x;
    float e, m;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fminf(x, 0.f) * 1.44269504f));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m) : "f"(x));  // NaN of NaN
    // (x > 0: x + 1)
    return m + e;
}
// phi' from phi: where phi > 1 the slope is 1, elsewhere phi itself.
__device__ __forceinline__ float slope_fast(float x, float f, int phi) {
    return !phi || x > 0.f ? 1.f : f;
}
__device__ __forceinline__ float low_of(unsigned u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_of(unsigned u) { return __uint_as_float(u & 0xffff0000u); }

// Four features of a row, of which n exist (the others 0), as bf16 pairs.
__device__ __forceinline__ uint2 load4(const T *x, int n, bool wide) {
    if (wide) return n > 0 ? *reinterpret_cast<const uint2 *>(x) : make_uint2(0, 0);
    const unsigned short *s = reinterpret_cast<const unsigned short *>(x);
    unsigned v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? s[i] : 0;
    return make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
}
__device__ __forceinline__ float4 load4(const float *x, int n, bool wide) {
    if (wide) return n > 0 ? *reinterpret_cast<const float4 *>(x) : make_float4(0, 0, 0, 0);
    return make_float4(n > 0 ? x[0] : 0.f, n > 1 ? x[1] : 0.f, n > 2 ? x[2] : 0.f,
                       n > 3 ? x[3] : 0.f);
}
__device__ __forceinline__ void open4(uint2 u, float (&e)[4]) {
    e[0] = low_of(u.x), e[1] = high_of(u.x), e[2] = low_of(u.y), e[3] = high_of(u.y);
}
__device__ __forceinline__ uint2 shut4(const float (&e)[4]) {
    return make_uint2(tc::pack_bf16x2(e[0], e[1]), tc::pack_bf16x2(e[2], e[3]));
}
// What e loses as bf16 (`high`), as bf16; 0 where that is not finite.
__device__ __forceinline__ uint2 rest4(const float (&e)[4], uint2 high) {
    float h[4], r[4];
    open4(high, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = fabsf(h[i]) < INFINITY ? e[i] - h[i] : 0.f;
    return shut4(r);
}

__device__ __forceinline__ void ldmatrix4(unsigned (&r)[4], const T *at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(tc::smem_u32(at)) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(unsigned (&r)[4], const T *at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(tc::smem_u32(at)) : "memory");
}
// c += a b, 16 x 16 times 16 x 8.
__device__ __forceinline__ void mma(float (&c)[4], const unsigned (&a)[4], unsigned b0,
                                    unsigned b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kPad = 8;  // features more per row of shared memory: no bank conflicts

// ---------------------------------------------------------------- sums of outer products

// S[a][c] += w_i f(x_i)[a] y_i[c] and z[a] += u_i w_i f(x_i)[a] over a part of the tokens
// (w = r or 1, u = -t or 1), 64 features a and all c per block, 32 x 32 per warp.
template <int kC>
__global__ void __launch_bounds__(2 * kC, kC == 256 ? 1 : 2) half_sum_kernel(const SumParams p,
                                                                             int wide) {
    constexpr int kT = 2 * kC, kA = 64, kTok = 32;
    constexpr int kX = kTok * kA / 4 / kT, kY = kTok * kC / 4 / kT;  // fours of a thread
    constexpr int kStepX = kT / (kA / 4), kStepY = kT / (kC / 4);    // rows apart
    __shared__ __align__(16) T Ah[kTok][kA + kPad], Al[kTok][kA + kPad], Y[kTok][kC + kPad];
    static_assert(sizeof(Y) >= sizeof(float) * kStepX * kA, "the threads' parts of z fit");
    const int tiles = (p.d + kA - 1) / kA;
    const long long head = blockIdx.x / tiles;
    const int a0 = (int)(blockIdx.x - head * tiles) * kA, seg = blockIdx.y;
    const int b = (int)(head / p.Hk), h = (int)(head % p.Hk);
    const int len = tokens_of(p.lengths, b, p.L);
    const long long all = (long long)p.group * p.L;
    const long long i0 = seg * p.per, i1 = min(i0 + p.per, all);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wa = (warp & 1) * 32, wc = (warp >> 1) * 32;
    const int fx = threadIdx.x % (kA / 4) * 4, rx = threadIdx.x / (kA / 4);
    const int fy = threadIdx.x % (kC / 4) * 4, ry = threadIdx.x / (kC / 4);
    const int nx = p.d - a0 - fx, ny = p.d - fy;  // features that exist from there on
    const T *xs = static_cast<const T *>(p.x) + b * p.sx.b + a0 + fx;
    const T *ys = static_cast<const T *>(p.y) + b * p.sy.b + fy;
    float acc[2][4][4] = {}, total[2][4][4] = {}, zacc[4] = {};
    uint2 x[kX], y[kY];
    float2 rt[kX];
    int g0 = (int)(i0 / max(p.L, 1)), n0 = (int)(i0 - (long long)g0 * p.L);  // of token i
    auto fetch = [&](long long i) {
        // where token i + row lies, if it is one
        auto place = [&](int row, int &g, int &n) {
            g = g0, n = n0 + row;
            if (n >= p.L) g += n / p.L, n %= p.L;
            return i + row < i1 && n < len;
        };
        if (i + kTok <= i1 && n0 + kTok <= min(p.L, len)) {  // rows of one head, all of them
            const long long hh = (long long)h * p.group + g0;
            const T *px = xs + hh * p.sx.h + (n0 + rx) * p.sx.n;
            const T *py = ys + hh * p.sy.h + (n0 + ry) * p.sy.n;
#pragma unroll
            for (int k = 0; k < kX; ++k) {
                rt[k] = p.rt ? p.rt[(head * p.group + g0) * p.L + n0 + rx + k * kStepX]
                             : make_float2(1.f, -1.f);
                x[k] = load4(px + k * kStepX * p.sx.n, nx, wide);
            }
#pragma unroll
            for (int k = 0; k < kY; ++k) y[k] = load4(py + k * kStepY * p.sy.n, ny, wide);
            n0 += kTok;
            if (n0 == p.L) ++g0, n0 = 0;
            return;
        }
        int g, n;
#pragma unroll
        for (int k = 0; k < kX; ++k) {
            const bool ok = place(rx + k * kStepX, g, n);
            const long long hh = (long long)h * p.group + g;
            rt[k] = make_float2(ok ? 1.f : 0.f, -1.f);
            if (ok && p.rt) rt[k] = p.rt[(head * p.group + g) * p.L + n];
            x[k] = make_uint2(0, 0);
            if (ok) x[k] = load4(xs + hh * p.sx.h + n * p.sx.n, nx, wide);
        }
#pragma unroll
        for (int k = 0; k < kY; ++k) {
            const bool ok = place(ry + k * kStepY, g, n);
            const long long hh = (long long)h * p.group + g;
            y[k] = make_uint2(0, 0);
            if (ok) y[k] = load4(ys + hh * p.sy.h + n * p.sy.n, ny, wide);
        }
        n0 += kTok;
        if (n0 >= p.L) g0 += n0 / p.L, n0 %= p.L;
    };
    auto fold = [&]() {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) total[m][j][e] += acc[m][j][e], acc[m][j][e] = 0.f;
    };
    const long long end = p.group == 1 ? min(i1, (long long)len) : i1;
    if (i0 < end) fetch(i0);
    int steps = 0;
    for (long long i = i0; i < end; i += kTok) {
        __syncthreads();
        bool none = false;
#pragma unroll
        for (int k = 0; k < kX; ++k) {
            const int row = rx + k * kStepX;
            const bool gone = is_none(rt[k]);
            const float u = gone ? 0.f : -rt[k].y;
            none |= gone;
            float e[4];
            open4(x[k], e);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                e[j] = j < nx ? rt[k].x * phi_fast(e[j], p.phi) : 0.f;
                zacc[j] = fmaf(e[j], u, zacc[j]);
            }
            const uint2 high = shut4(e);
            *reinterpret_cast<uint2 *>(&Ah[row][fx]) = high;
            *reinterpret_cast<uint2 *>(&Al[row][fx]) = rest4(e, high);
        }
#pragma unroll
        for (int k = 0; k < kY; ++k) *reinterpret_cast<uint2 *>(&Y[ry + k * kStepY][fy]) = y[k];
        if (__syncthreads_or(none)) {  // rows of 0 times what may not be finite
#pragma unroll
            for (int k = 0; k < kX; ++k)
                if (is_none(rt[k]))
                    for (int c = fx; c < kC; c += kA)
                        *reinterpret_cast<uint2 *>(&Y[rx + k * kStepX][c]) = make_uint2(0, 0);
            __syncthreads();
        }
        if (i + kTok < end) fetch(i + kTok);
#pragma unroll
        for (int ks = 0; ks < kTok; ks += 16) {
            unsigned u[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                ldmatrix4_t(u[j], &Y[ks + (lane & 15)][wc + 16 * j + (lane >> 4) * 8]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int k = ks + (lane >> 4) * 8 + (lane & 7),
                          a = wa + 16 * m + ((lane >> 3) & 1) * 8;
                unsigned v[4];
                ldmatrix4_t(v, &Ah[k][a]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma(acc[m][j], v, u[j >> 1][2 * (j & 1)], u[j >> 1][2 * (j & 1) + 1]);
                ldmatrix4_t(v, &Al[k][a]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma(acc[m][j], v, u[j >> 1][2 * (j & 1)], u[j >> 1][2 * (j & 1) + 1]);
            }
        }
        if (++steps % (256 / kTok) == 0) fold();
    }
    fold();
    float *S = p.S + (seg * p.heads + head) * p.d * p.d;
    float *z = p.z + (seg * p.heads + head) * p.d;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int a = a0 + wa + 16 * m + (lane >> 2) + (e >> 1) * 8;
                const int c = wc + 8 * j + (lane & 3) * 2 + (e & 1);
                if (a < p.d && c < p.d) S[a * p.d + c] = total[m][j][e];
            }
    // the threads' parts of z, in order
    __syncthreads();
    float *parts = reinterpret_cast<float *>(Y);
#pragma unroll
    for (int j = 0; j < 4; ++j) parts[rx * kA + fx + j] = zacc[j];
    __syncthreads();
    if (threadIdx.x < kA && a0 + (int)threadIdx.x < p.d) {
        float t = 0.f;
        for (int q = 0; q < kStepX; ++q) t += parts[q * kA + threadIdx.x];
        z[a0 + threadIdx.x] = t;
    }
}

// ---------------------------------------------------------------- rows times a state

constexpr int kRows = 128, kStep = 32;  // rows of a block, features of one staging

// A pair of results of a row, features c and c + 1 of d.
__device__ __forceinline__ void store2(T *row, int c, int d, float v0, float v1, bool words) {
    if (words) {
        if (c < d) *reinterpret_cast<unsigned *>(row + c) = tc::pack_bf16x2(v0, v1);
    } else {
        if (c < d) row[c] = __float2bfloat16_rn(v0);
        if (c + 1 < d) row[c + 1] = __float2bfloat16_rn(v1);
    }
}

// y_i = S^T f(x_i), over f . z with norm: 128 rows and all columns per block, 32 x 64 per
// warp.
template <int kC>
__global__ void __launch_bounds__(2 * kC, kC == 256 ? 1 : 2)
half_read_kernel(const ReadParams p, int wide, int wide_s, int words) {
    constexpr int kT = 2 * kC;
    constexpr int kX = kRows * kStep / 4 / kT, kS = kStep * kC / 4 / kT;
    __shared__ __align__(16) T A[kRows][kStep + kPad], Y[kStep][kC + kPad];
    __shared__ float rows_den[kRows];
    const int row_tiles = (p.L + kRows - 1) / kRows;
    const long long bh = blockIdx.x / row_tiles;  // of x's heads
    const int n0 = (int)(blockIdx.x - bh * row_tiles) * kRows;
    const int H = p.Hk * p.group, b = (int)(bh / H), h = (int)(bh % H);
    const long long state = (long long)b * p.Hk + h / p.group;
    const int len = tokens_of(p.lengths, b, p.L);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wr = (warp & 3) * 32, wc = (warp >> 2) * 64;
    const int fx = threadIdx.x % (kStep / 4) * 4, rx = threadIdx.x / (kStep / 4);
    const int fs = threadIdx.x % (kC / 4) * 4, rs = threadIdx.x / (kC / 4);
    const T *x = static_cast<const T *>(p.x) + b * p.sx.b + h * p.sx.h;
    const float *S = p.S + state * p.d * p.d, *z = p.z + state * p.d;
    float acc[2][8][4] = {}, den[kX] = {};
    uint2 xv[kX];
    float4 sv[kS];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int n = n0 + rx + i * (kT / (kStep / 4));
            xv[i] = make_uint2(0, 0);
            if (n < len) xv[i] = load4(x + n * p.sx.n + k0 + fx, p.d - k0 - fx, wide);
        }
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            const int a = k0 + rs + i * (kT / (kC / 4));
            sv[i] = load4(S + a * p.d + fs, a < p.d ? p.d - fs : 0, wide_s);
        }
    };
    fetch(0);
    for (int k0 = 0; k0 < p.d; k0 += kStep) {
        float zv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            zv[j] = p.norm && k0 + fx + j < p.d ? z[k0 + fx + j] : 0.f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            float e[4];
            open4(xv[i], e);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                e[j] = k0 + fx + j < p.d ? phi_fast(e[j], p.phi) : 0.f;
            const uint2 f = shut4(e);
            *reinterpret_cast<uint2 *>(&A[rx + i * (kT / (kStep / 4))][fx]) = f;
            open4(f, e);  // the denominator by the rounded ones, too
#pragma unroll
            for (int j = 0; j < 4; ++j) den[i] = fmaf(e[j], zv[j], den[i]);
        }
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            const float e[4] = {sv[i].x, sv[i].y, sv[i].z, sv[i].w};
            *reinterpret_cast<uint2 *>(&Y[rs + i * (kT / (kC / 4))][fs]) = shut4(e);
        }
        __syncthreads();
        if (k0 + kStep < p.d) fetch(k0 + kStep);
#pragma unroll
        for (int ks = 0; ks < kStep; ks += 16) {
            unsigned v[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
                ldmatrix4(v[m], &A[wr + 16 * m + (lane & 15)][ks + (lane >> 4) * 8]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                unsigned u[4];
                ldmatrix4_t(u, &Y[ks + (lane & 15)][wc + 16 * j + (lane >> 4) * 8]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma(acc[m][2 * j], v[m], u[0], u[1]);
                    mma(acc[m][2 * j + 1], v[m], u[2], u[3]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kX; ++i) {
#pragma unroll
        for (int o = 1; o < kStep / 4; o <<= 1) den[i] += __shfl_xor_sync(~0u, den[i], o);
        if (fx == 0) rows_den[rx + i * (kT / (kStep / 4))] = p.norm ? den[i] : 1.f;
    }
    __syncthreads();
    T *y = static_cast<T *>(p.y) + b * p.sy.b + h * p.sy.h;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = wr + 16 * m + 8 * i + (lane >> 2), n = n0 + row;
            if (n >= p.L) continue;
            // Without keys there is nothing to average: 0.  (The sign for that is the
            // denominator itself: 1 / den is 0 for an infinite one, too.)
            const float d = rows_den[row], inv = 1.f / d;
            const bool ok = n < len && d != 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                store2(y + n * p.sy.n, wc + 8 * j + (lane & 3) * 2, p.d,
                       ok ? acc[m][j][2 * i] * inv : 0.f,
                       ok ? acc[m][j][2 * i + 1] * inv : 0.f, words);
        }
}

// G_i = S y_i, and from it the gradient of row i: on q's side r (G - t z) phi'(x) with r
// and t left for the sums, on k's side (G + z) phi'(x) (z is then dz).  128 rows and all
// features per block, 32 x 64 per warp.
template <int kC>
struct GradSmem {
    T Wh[kC][kStep + kPad], Wl[kC][kStep + kPad], Y[kRows][kStep + kPad];
    float2 red[kC / 64][kRows];  // f . G and f . z of a row, of 64 features each
    float2 z[kC / 2];            // 0 where it is not used
};

template <int kC>
__global__ void __launch_bounds__(2 * kC, kC == 256 ? 1 : 2)
half_grad_kernel(const GradParams p, int wide, int wide_s, int words) {
    constexpr int kT = 2 * kC;
    constexpr int kX = kRows * kStep / 4 / kT, kS = kC * kStep / 4 / kT;
    constexpr int kApart = kT / (kStep / 4);
    extern __shared__ __align__(16) uint8_t raw[];
    GradSmem<kC> &sm = *reinterpret_cast<GradSmem<kC> *>(raw);
    const int row_tiles = (p.L + kRows - 1) / kRows;
    const long long bh = blockIdx.x / row_tiles;
    const int n0 = (int)(blockIdx.x - bh * row_tiles) * kRows;
    const int H = p.Hk * p.group, b = (int)(bh / H), h = (int)(bh % H);
    const long long state = (long long)b * p.Hk + h / p.group;
    const int len = tokens_of(p.lengths, b, p.L);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wr = (warp & 3) * 32, wa = (warp >> 2) * 64;
    const int f0 = threadIdx.x % (kStep / 4) * 4, r0 = threadIdx.x / (kStep / 4);
    const T *y = static_cast<const T *>(p.y) + b * p.sy.b + h * p.sy.h;
    const T *x = static_cast<const T *>(p.x) + b * p.sx.b + h * p.sx.h;
    const float *S = p.S + state * p.d * p.d, *z = p.z + state * p.d;
    float acc[2][8][4] = {};
    uint2 yv[kX];
    float4 sv[kS];
    auto fetch = [&](int k0) {
        const int rest = p.d - k0 - f0;
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int n = n0 + r0 + i * kApart;
            yv[i] = make_uint2(0, 0);
            if (n < len) yv[i] = load4(y + n * p.sy.n + k0 + f0, rest, wide);
        }
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            const int a = r0 + i * kApart;
            sv[i] = load4(S + a * p.d + k0 + f0, a < p.d ? rest : 0, wide_s);
        }
    };
    fetch(0);
    if (threadIdx.x < kC)
        reinterpret_cast<float *>(sm.z)[threadIdx.x] =
            (p.norm || p.keys) && (int)threadIdx.x < p.d ? z[threadIdx.x] : 0.f;
    for (int k0 = 0; k0 < p.d; k0 += kStep) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kX; ++i)
            *reinterpret_cast<uint2 *>(&sm.Y[r0 + i * kApart][f0]) = yv[i];
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            const float e[4] = {sv[i].x, sv[i].y, sv[i].z, sv[i].w};
            const uint2 high = shut4(e);
            *reinterpret_cast<uint2 *>(&sm.Wh[r0 + i * kApart][f0]) = high;
            *reinterpret_cast<uint2 *>(&sm.Wl[r0 + i * kApart][f0]) = rest4(e, high);
        }
        __syncthreads();
        if (k0 + kStep < p.d) fetch(k0 + kStep);
#pragma unroll
        for (int ks = 0; ks < kStep; ks += 16) {
            unsigned v[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
                ldmatrix4(v[m], &sm.Y[wr + 16 * m + (lane & 15)][ks + (lane >> 4) * 8]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int a = wa + 16 * j + (lane & 7) + (lane >> 4) * 8,
                          c = ks + ((lane >> 3) & 1) * 8;
                unsigned u[4];
                ldmatrix4(u, &sm.Wh[a][c]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma(acc[m][2 * j], v[m], u[0], u[1]);
                    mma(acc[m][2 * j + 1], v[m], u[2], u[3]);
                }
                ldmatrix4(u, &sm.Wl[a][c]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma(acc[m][2 * j], v[m], u[0], u[1]);
                    mma(acc[m][2 * j + 1], v[m], u[2], u[3]);
                }
            }
        }
    }
    // features a and a + 1 of a row of x, and z there
    auto pair_of = [&](const T *row, int a) {
        if (words) return a < p.d ? *reinterpret_cast<const unsigned *>(row + a) : 0u;
        const unsigned short *s = reinterpret_cast<const unsigned short *>(row);
        return (a < p.d ? s[a] : 0u) | (a + 1 < p.d ? (unsigned)s[a + 1] << 16 : 0u);
    };
    if (!p.keys) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = wr + 16 * m + 8 * i + (lane >> 2), n = n0 + row;
                float dot = 0.f, den = 0.f;
                if (n < len)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int a = wa + 8 * j + (lane & 3) * 2;
                        if (a >= p.d) continue;
                        const unsigned u = pair_of(x + n * p.sx.n, a);
                        const float e0 = phi_fast(low_of(u), p.phi);
                        const float e1 = a + 1 < p.d ? phi_fast(high_of(u), p.phi) : 0.f;
                        dot = fmaf(e0, acc[m][j][2 * i], fmaf(e1, acc[m][j][2 * i + 1], dot));
                        const float2 za = sm.z[a / 2];
                        den = fmaf(e0, za.x, fmaf(e1, za.y, den));
                    }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    dot += __shfl_xor_sync(~0u, dot, o);
                    den += __shfl_xor_sync(~0u, den, o);
                }
                if ((lane & 3) == 0) sm.red[warp >> 2][row] = make_float2(dot, den);
            }
        __syncthreads();
    }
    T *dx = static_cast<T *>(p.dx) + b * p.sdx.b + h * p.sdx.h;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = wr + 16 * m + 8 * i + (lane >> 2), n = n0 + row;
            if (n >= p.L) continue;
            float r = 1.f, t = p.keys ? -1.f : 0.f;
            bool none = false;
            if (!p.keys) {
                float dot = 0.f, den = 0.f;
#pragma unroll
                for (int q = 0; q < kC / 64; ++q)
                    dot += sm.red[q][row].x, den += sm.red[q][row].y;
                if (p.norm) {
                    none = den == 0.f;
                    r = none ? 0.f : 1.f / den;
                    t = dot * r;
                }
                if (wa == 0 && (lane & 3) == 0)
                    p.rt[bh * p.L + n] = none ? no_row() : make_float2(r, t);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int a = wa + 8 * j + (lane & 3) * 2;
                if (a >= p.d) continue;
                float g[2] = {};
                if (n < len && !none) {
                    const unsigned u = pair_of(x + n * p.sx.n, a);
                    const float2 za = sm.z[a / 2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float xe = e ? high_of(u) : low_of(u);
                        g[e] = r * fmaf(-t, e ? za.y : za.x, acc[m][j][2 * i + e]) *
                               slope_fast(xe, phi_fast(xe, p.phi), p.phi);
                    }
                }
                store2(dx + n * p.sdx.n, a, p.d, g[0], g[1], words);
            }
        }
}

// ---------------------------------------------------------------- launches

// Whether all rows start at a multiple of `bytes`, and have such a size.
bool aligned(const void *x, const la_strides &s, int d, int bytes) {
    const unsigned long long all = (unsigned long long)(uintptr_t)x | (unsigned)d * 2u |
                                   (unsigned long long)s.b * 2 | (unsigned long long)s.h * 2 |
                                   (unsigned long long)s.n * 2;
    return all % bytes == 0;
}
bool aligned_states(const float *S, int d) { return (uintptr_t)S % 16 == 0 && d % 4 == 0; }

template <typename F>
cudaError_t by_width(int d, F &&go) {
    if (d <= 64) return go(std::integral_constant<int, 64>());
    if (d <= 128) return go(std::integral_constant<int, 128>());
    return go(std::integral_constant<int, 256>());
}

cudaError_t counted() {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) note_launches(1);
    return e;
}

}  // namespace

cudaError_t half_sums(const SumParams &p, cudaStream_t s) {
    const int wide = aligned(p.x, p.sx, p.d, 8) && aligned(p.y, p.sy, p.d, 8);
    return by_width(p.d, [&](auto c) {
        const dim3 grid((unsigned)(p.heads * ((p.d + 63) / 64)), (unsigned)p.segs);
        half_sum_kernel<c.value><<<grid, 2 * c.value, 0, s>>>(p, wide);
        return counted();
    });
}

cudaError_t half_read(const ReadParams &p, long long heads, cudaStream_t s) {
    const long long blocks = heads * (((long long)p.L + kRows - 1) / kRows);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const int wide = aligned(p.x, p.sx, p.d, 8), wide_s = aligned_states(p.S, p.d),
              words = aligned(p.y, p.sy, p.d, 4);
    return by_width(p.d, [&](auto c) {
        half_read_kernel<c.value><<<(unsigned)blocks, 2 * c.value, 0, s>>>(p, wide, wide_s, words);
        return counted();
    });
}

cudaError_t half_grads(const GradParams &p, long long heads, cudaStream_t s) {
    const long long blocks = heads * (((long long)p.L + kRows - 1) / kRows);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const int wide = aligned(p.y, p.sy, p.d, 8), wide_s = aligned_states(p.S, p.d),
              words = aligned(p.x, p.sx, p.d, 4) && aligned(p.dx, p.sdx, p.d, 4);
    return by_width(p.d, [&](auto c) {
        constexpr int smem = (int)sizeof(GradSmem<c.value>);
        const cudaError_t e = cudaFuncSetAttribute(
            half_grad_kernel<c.value>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        half_grad_kernel<c.value><<<(unsigned)blocks, 2 * c.value, smem, s>>>(p, wide, wide_s, words);
        return counted();
    });
}

}  // namespace cross
}  // namespace la

// Norms of queries and keys per head and their position rotation, forward and
// backward (la_qk_norm_rope, la_backward_qk_norm_rope in include/linattn.h).
//
// A row x (one token of one head, d values) becomes
//   n = x r, r = 1 / sqrt(mean(x^2) + eps),  u = w n,
//   (y1, y2) = (u1 cos t - u2 sin t, u2 cos t + u1 sin t)  for each pair;
// backwards, with g the output's gradient turned by -t,
//   dw = sum_rows g n,   dx = r (w g - n mean(n w g)).
//
// The angle t = p f of position p and frequency f (radians) is held as a
// fraction of a turn in 64-bit fixed point: f / 2 pi mod 1 is rounded to
// 2^-64 on the host, and p times that wraps modulo one turn exactly, so an
// angle far out costs one integer product and loses nothing.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "la_internal.h"
#include "la_tc.h"
#include "la_tc_host.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = LA_MAX_D / 2;

// One side (queries or keys) of a call.  Strides are in elements.
struct Side {
    const void *x;   // forward input (backward: may be NULL without norm)
    const void *dy;  // backward: gradient of the output
    void *y;         // forward: output; backward: gradient of the input
    const void *w;   // weight or NULL
    float *dw;       // backward: weight gradient or NULL
    la_strides sx, sdy, sy;
    int H;
};

struct Params {
    Side side[2];
    const void *positions;
    long long pos_b, pos_n, offset;
    int pos_bytes;
    int B, N, d, half, interleaved, norm, w_bf16;
    float eps, inv_d;
    float *partial;  // backward: a row of d sums of g n for each block, or NULL
    // the split of the work, see qk_rows_kernel
    int lane_bits, token_bits, heads_per_unit, chunks[2], blocks_q;
    unsigned long long turns[kMaxPairs];  // frequency, 2^-64 turns per position
};

// V values of T as they lie in memory: one load or store of V * sizeof(T) bytes.
template <int kBytes> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = unsigned; };
template <> struct Raw<2> { using type = unsigned short; };

template <typename T, int V>
struct Pack {
    union {
        typename Raw<sizeof(T) * V>::type raw;
        T v[V];
    };
    __device__ Pack() {}
};
template <typename T, int V>
__device__ __forceinline__ void load(Pack<T, V> &p, const T *src) {
    p.raw = *reinterpret_cast<const typename Raw<sizeof(T) * V>::type *>(src);
}
template <typename T, int V>
__device__ __forceinline__ void store(T *dst, const Pack<T, V> &p) {
    *reinterpret_cast<typename Raw<sizeof(T) * V>::type *>(dst) = p.raw;
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float &d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float x) { d = __float2bfloat16_rn(x); }

__device__ __forceinline__ float weight_at(const void *w, int w_bf16, int i) {
    if (!w) return 1.f;
    return w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i])
                  : static_cast<const float *>(w)[i];
}

__device__ __forceinline__ long long position_of(const Params &p, int b, int n) {
    if (!p.positions) return n + p.offset;
    const long long i = b * p.pos_b + n * p.pos_n;
    const long long v = p.pos_bytes == 8 ? static_cast<const long long *>(p.positions)[i]
                                         : static_cast<const int *>(p.positions)[i];
    return v + p.offset;
}

// cos and sin of pos * turns (2^-64 turns).  The top 32 bits as a signed
// number are the angle in 2^-31 half turns, in [-1, 1).
__device__ __forceinline__ void turn_of(long long pos, unsigned long long turns, float *c,
                                        float *s) {
    const unsigned long long phase = (unsigned long long)pos * turns;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, s, c);
}

// Sum over a row of K chunks of V terms in each of 2^bits lanes.  Term e of
// chunk j in lane l stands for pair ((j << bits) + l) V + e; the sum is the
// binary tree over the pair's bits from the lowest up, so that it does not
// depend on V: a row gives the same bits whatever its alignment.
template <int V, int K>
__device__ __forceinline__ float row_sum(float (&t)[K][V], int bits) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
        for (int o = 1; o < V; o *= 2)
#pragma unroll
            for (int e = 0; e < V; e += 2 * o) t[j][e] += t[j][e + o];
        for (int o = 1; o >> bits == 0; o <<= 1) t[j][0] += __shfl_xor_sync(~0u, t[j][0], o);
    }
#pragma unroll
    for (int o = 1; o < K; o *= 2)
#pragma unroll
        for (int j = 0; j < K; j += 2 * o) t[j][0] += t[j + o][0];
    return t[0][0];
}

// A row is shared by 2^lane_bits lanes of a warp.  A lane takes K chunks of V
// pairs, each as two vectors of V values: (lo, hi) = features (2i, 2i + V)
// where pairs are neighbours (kInter, and where d is odd, which leaves the last
// alone), else (i, i + half) in the rotated part and (i + half, i + d / 2) in
// the rest: both values of a pair are always in one thread and every access is
// one vector.  A block's groups of lanes are 2^token_bits tokens
// times as many heads as are left; a unit of work is such a tile of tokens and
// `heads_per_unit` heads of one side.  Angles (a 64-bit product, sincospi) are
// formed once per token and lane and serve all heads of the unit.
//
// Forward: one unit per block.  Backward: a block takes the units of one side
// blockIdx, blockIdx + blocks, ..., and keeps its sums of g n in registers; they
// leave once at its end.
template <typename T, int V, int K, bool kInter, bool kBack>
__global__ void __launch_bounds__(kThreads) qk_rows_kernel(const __grid_constant__ Params p) {
    constexpr int U = kBack ? (V == 1 ? 1 : 2) : (V * K >= 8 ? 2 : 4);  // rows in flight
    const int bits = p.lane_bits, lane = threadIdx.x & ((1 << bits) - 1);
    const int group = threadIdx.x >> bits;
    const int tok_in = group & ((1 << p.token_bits) - 1), head_in = group >> p.token_bits;
    const int head_step = (kThreads >> bits) >> p.token_bits;
    const int pairs = (p.d + 1) / 2;
    const long long tokens = (long long)p.B * p.N;

    int which;
    long long unit, unit_step;
    if (kBack) {
        which = (int)blockIdx.x >= p.blocks_q;
        unit = which ? blockIdx.x - p.blocks_q : blockIdx.x;
        unit_step = which ? gridDim.x - p.blocks_q : p.blocks_q;
    } else {
        const int all = p.chunks[0] + p.chunks[1];
        const long long tile = blockIdx.x / all;
        const int chunk = (int)(blockIdx.x - tile * all);
        which = chunk >= p.chunks[0];
        unit = tile * p.chunks[which] + (which ? chunk - p.chunks[0] : chunk);
        unit_step = 0;
    }
    const Side &sd = p.side[which];
    const int chunks = p.chunks[which], H = sd.H;
    const long long units = ((tokens + (1 << p.token_bits) - 1) >> p.token_bits) * chunks;

    // this lane's features and their weights
    int lo[K], hi[K];
    bool l_ok[K], h_ok[K];
    float w[K][2 * V];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int i = (lane + (j << bits)) * V;  // first pair of the chunk
        const bool rot = i < p.half, next = kInter || (!rot && p.d % 2);
        lo[j] = next ? 2 * i : rot ? i : i + p.half;
        hi[j] = next ? 2 * i + V : rot ? i + p.half : i + p.d / 2;
        l_ok[j] = i < pairs;
        h_ok[j] = l_ok[j] && hi[j] < p.d;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[j][e] = l_ok[j] ? weight_at(sd.w, p.w_bf16, lo[j] + e) : 0.f;
            w[j][V + e] = h_ok[j] ? weight_at(sd.w, p.w_bf16, hi[j] + e) : 0.f;
        }
    }
    float dw[K][2 * V] = {};

    do {
        const long long tile = unit / chunks;
        const int h0 = (int)(unit - tile * chunks) * p.heads_per_unit;
        const int h1 = min(h0 + p.heads_per_unit, H);
        const long long tok = (tile << p.token_bits) + tok_in;
        const bool t_ok = tok < tokens && (!kBack || unit < units);
        const bool small = tokens <= 0x7fffffff;
        const int b = !t_ok ? 0 : small ? (int)((unsigned)tok / (unsigned)p.N) : (int)(tok / p.N);
        const int n = t_ok ? (int)(tok - (long long)b * p.N) : 0;
        const T *x = static_cast<const T *>(sd.x) + b * sd.sx.b + n * sd.sx.n;
        const T *dy = static_cast<const T *>(sd.dy) + b * sd.sdy.b + n * sd.sdy.n;
        T *y = static_cast<T *>(sd.y) + b * sd.sy.b + n * sd.sy.n;

        float cs[K][V], sn[K][V];
        const long long pos = p.half && t_ok ? position_of(p, b, n) : 0;
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int i = (lane + (j << bits)) * V + e;
                cs[j][e] = 1.f;
                sn[j][e] = 0.f;
                if (i < p.half) turn_of(pos, p.turns[i], &cs[j][e], &sn[j][e]);
            }

        for (int h = h0 + head_in; h - head_in < h1; h += U * head_step) {
            Pack<T, V> rx[U][K][2], rg[U][K][2];
            bool ok[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hu = h + u * head_step;
                ok[u] = t_ok && hu < h1;
                if (!ok[u]) continue;
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    if (!kBack || p.norm) {
                        if (l_ok[j]) load<T, V>(rx[u][j][0], x + hu * sd.sx.h + lo[j]);
                        if (h_ok[j]) load<T, V>(rx[u][j][1], x + hu * sd.sx.h + hi[j]);
                    }
                    if (kBack) {
                        if (l_ok[j]) load<T, V>(rg[u][j][0], dy + hu * sd.sdy.h + lo[j]);
                        if (h_ok[j]) load<T, V>(rg[u][j][1], dy + hu * sd.sdy.h + hi[j]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[K][2 * V], g[K][2 * V];
                float ss[K][V], dot[K][V];
#pragma unroll
                for (int j = 0; j < K; ++j) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const bool have = ok[u] && (!kBack || p.norm);
                        v[j][e] = have && l_ok[j] ? to_f(rx[u][j][0].v[e]) : 0.f;
                        v[j][V + e] = have && h_ok[j] ? to_f(rx[u][j][1].v[e]) : 0.f;
                        if (kBack) {
                            g[j][e] = ok[u] && l_ok[j] ? to_f(rg[u][j][0].v[e]) : 0.f;
                            g[j][V + e] = ok[u] && h_ok[j] ? to_f(rg[u][j][1].v[e]) : 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int i0 = kInter ? 2 * e : e, i1 = kInter ? 2 * e + 1 : V + e;
                        ss[j][e] = fmaf(v[j][i0], v[j][i0], __fmul_rn(v[j][i1], v[j][i1]));
                        if (kBack) {
                            const float a = g[j][i0], c = g[j][i1];
                            g[j][i0] = fmaf(a, cs[j][e], __fmul_rn(c, sn[j][e]));
                            g[j][i1] = fmaf(c, cs[j][e], -__fmul_rn(a, sn[j][e]));
                            dot[j][e] = fmaf(__fmul_rn(v[j][i0], w[j][i0]), g[j][i0],
                                             __fmul_rn(__fmul_rn(v[j][i1], w[j][i1]), g[j][i1]));
                        }
                    }
                }
                float r = 1.f, m = 0.f;
                if (p.norm) {
                    r = rsqrtf(fmaf(row_sum<V, K>(ss, bits), p.inv_d, p.eps));
                    if (kBack)
                        m = __fmul_rn(__fmul_rn(row_sum<V, K>(dot, bits), p.inv_d),
                                      __fmul_rn(r, r));
                }
                const int hu = h + u * head_step;
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    Pack<T, V> o[2];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int i0 = kInter ? 2 * e : e, i1 = kInter ? 2 * e + 1 : V + e;
                        float o0, o1;
                        if (!kBack) {
                            const float a = __fmul_rn(__fmul_rn(v[j][i0], r), w[j][i0]);
                            const float c = __fmul_rn(__fmul_rn(v[j][i1], r), w[j][i1]);
                            o0 = fmaf(a, cs[j][e], -__fmul_rn(c, sn[j][e]));
                            o1 = fmaf(c, cs[j][e], __fmul_rn(a, sn[j][e]));
                        } else {
                            dw[j][i0] = fmaf(g[j][i0], __fmul_rn(v[j][i0], r), dw[j][i0]);
                            dw[j][i1] = fmaf(g[j][i1], __fmul_rn(v[j][i1], r), dw[j][i1]);
                            o0 = __fmul_rn(r, fmaf(w[j][i0], g[j][i0], -__fmul_rn(v[j][i0], m)));
                            o1 = __fmul_rn(r, fmaf(w[j][i1], g[j][i1], -__fmul_rn(v[j][i1], m)));
                        }
                        from_f(i0 < V ? o[0].v[i0 % V] : o[1].v[i0 % V], o0);
                        from_f(i1 < V ? o[0].v[i1 % V] : o[1].v[i1 % V], o1);
                    }
                    if (ok[u] && l_ok[j]) store<T, V>(y + hu * sd.sy.h + lo[j], o[0]);
                    if (ok[u] && h_ok[j]) store<T, V>(y + hu * sd.sy.h + hi[j], o[1]);
                }
            }
        }
        unit += unit_step;
    } while (kBack && unit < units);

    if (!kBack || !sd.dw) return;
    // the block's sums: over the groups of each warp, then over the warps
    __shared__ float sum[kThreads / 32][LA_MAX_D];
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) {
            float t = dw[j][e];
            for (int o = 1 << bits; o < 32; o <<= 1) t += __shfl_xor_sync(~0u, t, o);
            const int f = e < V ? lo[j] + e : hi[j] + e - V;
            if ((threadIdx.x & 31) == lane && (e < V ? l_ok[j] : h_ok[j])) sum[warp][f] = t;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += kThreads) {
        float t = 0.f;
        for (int q = 0; q < kThreads / 32; ++q) t += sum[q][i];
        p.partial[(long long)blockIdx.x * p.d + i] = t;
    }
}

// dw[i] = the sum of the blocks' partial sums: 1024 / 256 interleaved sums per
// feature, joined in order.
__global__ void __launch_bounds__(1024)
qk_weight_kernel(const float *partial, int blocks_q, int blocks, int d, float *dwq, float *dwk) {
    float *dw = blockIdx.x ? dwk : dwq;
    if (!dw) return;
    __shared__ float sum[4][LA_MAX_D];
    const int i = threadIdx.x & 255, part = threadIdx.x >> 8;
    const int b0 = blockIdx.x ? blocks_q : 0, b1 = blockIdx.x ? blocks : blocks_q;
    float t = 0.f;
    if (i < d) {
#pragma unroll 8
        for (int b = b0 + part; b < b1; b += 4) t += partial[(long long)b * d + i];
        sum[part][i] = t;
    }
    __syncthreads();
    if (part == 0 && i < d) dw[i] = ((sum[0][i] + sum[1][i]) + sum[2][i]) + sum[3][i];
}

la_status qk_fail(la_status s, const char *who, const char *msg) {
    char text[200];
    std::snprintf(text, sizeof(text), "%s: %s", who, msg);
    set_last_error(text);
    return s;
}

// Whether no two rows of d elements overlap.
bool rows_disjoint(const la_strides &s, int B, int H, int N, int d) {
    long long st[3] = {s.b, s.h, s.n}, ex[3] = {B, H, N};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (st[j] > st[j + 1]) {
                std::swap(st[j], st[j + 1]);
                std::swap(ex[j], ex[j + 1]);
            }
    long long span = d;  // elements from the first row's start to the last one's end
    for (int i = 0; i < 3; ++i) {
        if (ex[i] <= 1) continue;
        if (st[i] < span) return false;
        span += st[i] * (ex[i] - 1);
    }
    return true;
}

// f / (2 pi) mod 1 in 2^-64 turns.  1 / (2 pi) is the sum of two doubles, so
// the product is good to about 2^-64 turns for |f| up to a few turns.
unsigned long long turns_of(double f) {
    const double c = 0.15915494309189535, c_low = -9.839338337591243e-18;
    const double t = f * c;
    const double low = std::fma(f, c, -t) + f * c_low;  // |low| < 2^-51 |t|
    const double part = t - std::floor(t);              // exact, in [0, 1)
    const double top = std::floor(part * 0x1p32);
    const double rest = part * 0x1p32 - top;
    return ((unsigned long long)top << 32) + (unsigned long long)(rest * 0x1p32) +
           (unsigned long long)(long long)std::nearbyint((low - std::floor(low + 0.5)) * 0x1p64);
}

bool same(const la_strides &a, const la_strides &b) {
    return a.b == b.b && a.h == b.h && a.n == b.n;
}

bool aligned(const void *p, const la_strides &s, int B, int H, int N, int v, int elem) {
    return (uintptr_t)p % (uintptr_t)(v * elem) == 0 && (B <= 1 || s.b % v == 0) &&
           (H <= 1 || s.h % v == 0) && (N <= 1 || s.n % v == 0);
}

// Values per access: the most (up to `most`) that divide the row's two halves
// and its rotated part and at which every row of every tensor is aligned.
int vector_of(const Params &p, int most, int elem) {
    for (int v = most; v > 1; v /= 2) {
        bool ok = p.d % (2 * v) == 0 && p.half % v == 0;
        for (const Side &s : p.side)
            if (s.H > 0)
                ok = ok && aligned(s.x, s.sx, p.B, s.H, p.N, v, elem) &&
                     aligned(s.dy, s.sdy, p.B, s.H, p.N, v, elem) &&
                     aligned(s.y, s.sy, p.B, s.H, p.N, v, elem);
        if (ok) return v;
    }
    return 1;
}

template <typename T, int V, int K, bool kBack>
cudaError_t launch_rows(const Params &p, unsigned blocks, cudaStream_t stream) {
    if (p.interleaved)
        qk_rows_kernel<T, V, K, true, kBack><<<blocks, kThreads, 0, stream>>>(p);
    else
        qk_rows_kernel<T, V, K, false, kBack><<<blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, bool kBack>
la_status launch(const char *who, Params &p, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e != cudaSuccess) return qk_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    // 16-byte accesses forward; backward 4 values, so that the sums, weights
    // and angles of a lane leave room for enough warps
    const int most = kBack ? 4 : 16 / (int)sizeof(T);
    const int v = vector_of(p, most, (int)sizeof(T));
    const int chunks = ((p.d + 1) / 2 + v - 1) / v;  // of a row
    while ((1 << p.lane_bits) < chunks && p.lane_bits < 5) ++p.lane_bits;
    const int groups = kThreads >> p.lane_bits;
    const long long tokens = (long long)p.B * p.N;
    while ((1 << p.token_bits) < groups && (1 << p.token_bits) < tokens) ++p.token_bits;
    const int head_step = groups >> p.token_bits;
    const long long tiles = (tokens + (1 << p.token_bits) - 1) >> p.token_bits;
    // 8 heads per angle, fewer where that leaves SMs without work
    long long units = 0;
    for (int reuse = 8;; reuse /= 2) {
        p.heads_per_unit = head_step * reuse;
        units = 0;
        for (int i = 0; i < 2; ++i) {
            p.chunks[i] = (p.side[i].H + p.heads_per_unit - 1) / p.heads_per_unit;
            units += tiles * p.chunks[i];
        }
        if (reuse == 1 || units >= 4LL * sms) break;
    }
    long long blocks = units;
    if (kBack) {
        // as many blocks as run at once, shared by the sides as their units
        const long long most_blocks = 3LL * sms;
        const long long uq = tiles * p.chunks[0], uk = tiles * p.chunks[1];
        long long bq = uq, bk = uk;
        if (units > most_blocks) {
            bq = uq ? std::max(1LL, most_blocks * uq / units) : 0;
            bk = uk ? std::max(1LL, most_blocks - bq) : 0;
        }
        p.blocks_q = (int)bq;
        blocks = bq + bk;
    }
    if (blocks > 2147483647LL) return qk_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
    void *ws = nullptr;
    const bool want_dw = kBack && (p.side[0].dw || p.side[1].dw);
    if (want_dw) {
        e = tc_workspace_alloc(&ws, sizeof(float) * (size_t)blocks * p.d, stream);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return qk_fail(LA_ERR_NO_MEMORY, who, "workspace allocation");
        }
        p.partial = static_cast<float *>(ws);
    }
    constexpr int kV16 = 16 / (int)sizeof(T);
    if (!kBack && v == kV16 && kV16 == 8)
        e = launch_rows<T, kBack ? 4 : kV16, 1, kBack>(p, (unsigned)blocks, stream);
    else if (v == 4)
        e = launch_rows<T, 4, 1, kBack>(p, (unsigned)blocks, stream);
    else if (v == 2)
        e = launch_rows<T, 2, 2, kBack>(p, (unsigned)blocks, stream);
    else
        e = launch_rows<T, 1, 4, kBack>(p, (unsigned)blocks, stream);
    if (e == cudaSuccess) note_launches(1);
    if (e == cudaSuccess && want_dw) {
        qk_weight_kernel<<<2, 1024, 0, stream>>>(p.partial, p.blocks_q, (int)blocks, p.d,
                                                 p.side[0].dw, p.side[1].dw);
        e = cudaGetLastError();
        if (e == cudaSuccess) note_launches(1);
    }
    if (ws) {
        const cudaError_t ef = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e == cudaSuccess ? LA_OK : qk_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
}

// Checks shared by both directions; fills everything but the tensors.
la_status qk_common(const char *who, Params &p, const void *q_weight, const void *k_weight,
                    int norm, float eps, const la_rope *rope, int B, int Hq, int Hk, int N, int d,
                    la_dtype dtype, la_dtype weight_dtype) {
    if (B < 0 || N < 0 || Hq < 0 || Hk < 0)
        return qk_fail(LA_ERR_INVALID_ARG, who, "negative B, Hq, Hk or N");
    if (d < 1 || d > LA_MAX_D) return qk_fail(LA_ERR_INVALID_ARG, who, "d must be in 1..256");
    if (dtype != LA_F32 && dtype != LA_BF16)
        return qk_fail(LA_ERR_INVALID_ARG, who, "unknown dtype");
    if (norm != 0 && norm != 1) return qk_fail(LA_ERR_INVALID_ARG, who, "norm must be 0 or 1");
    if (norm && !(eps > 0.f && std::isfinite(eps)))
        return qk_fail(LA_ERR_INVALID_ARG, who, "eps must be positive and finite");
    if (!norm && (q_weight || k_weight))
        return qk_fail(LA_ERR_INVALID_ARG, who, "weights need norm");
    if ((q_weight || k_weight) && weight_dtype != LA_F32 && weight_dtype != LA_BF16)
        return qk_fail(LA_ERR_INVALID_ARG, who, "unknown weight dtype");
    if ((double)B * N * ((double)Hq + Hk) > 1e15)
        return qk_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
    p = Params{};
    p.B = B;
    p.N = N;
    p.d = d;
    p.norm = norm;
    p.eps = eps;
    p.inv_d = 1.f / (float)d;
    p.w_bf16 = weight_dtype == LA_BF16;
    p.side[0].H = Hq;
    p.side[1].H = Hk;
    p.side[0].w = q_weight;
    p.side[1].w = k_weight;
    if (!rope) return LA_OK;
    const int R = rope->rotary_dim;
    if (R < 0 || R > d || R % 2)
        return qk_fail(LA_ERR_INVALID_ARG, who, "rotary_dim must be even and in 0..d");
    if (rope->interleaved != 0 && rope->interleaved != 1)
        return qk_fail(LA_ERR_INVALID_ARG, who, "interleaved must be 0 or 1");
    if (R == 0) return LA_OK;
    if (!rope->frequencies) return qk_fail(LA_ERR_INVALID_ARG, who, "null frequencies");
    if (rope->positions) {
        if (rope->position_bytes != 4 && rope->position_bytes != 8)
            return qk_fail(LA_ERR_INVALID_ARG, who, "position_bytes must be 4 or 8");
        if (rope->position_stride_b < 0 || rope->position_stride_n < 0)
            return qk_fail(LA_ERR_INVALID_ARG, who, "negative position stride");
        if ((uintptr_t)rope->positions % (uintptr_t)rope->position_bytes)
            return qk_fail(LA_ERR_INVALID_ARG, who, "unaligned positions");
    }
    for (int i = 0; i < R / 2; ++i) {
        const double f = rope->frequencies[i];
        if (!(std::fabs(f) <= 1e9))  // also rejects NaN
            return qk_fail(LA_ERR_INVALID_ARG, who, "frequencies must lie in [-1e9, 1e9]");
        p.turns[i] = turns_of(f);
    }
    p.half = R / 2;
    p.interleaved = rope->interleaved;
    p.positions = rope->positions;
    p.pos_bytes = rope->position_bytes;
    p.pos_b = rope->position_stride_b;
    p.pos_n = rope->position_stride_n;
    p.offset = rope->offset;
    return LA_OK;
}

la_strides contiguous(int H, int N, int d) {
    return {(long long)H * N * d, (long long)N * d, d};
}

bool negative(const la_strides &s) { return s.b < 0 || s.h < 0 || s.n < 0; }

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

__attribute__((visibility("default")))
la_status la_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out,
                          const la_strides *strides, const void *q_weight, const void *k_weight,
                          int norm, float eps, const la_rope *rope, int B, int Hq, int Hk, int N,
                          int d, la_dtype dtype, la_dtype weight_dtype, la_stream_t stream) {
    const char *who = "la_qk_norm_rope";
    Params p;
    la_status st = qk_common(who, p, q_weight, k_weight, norm, eps, rope, B, Hq, Hk, N, d, dtype,
                             weight_dtype);
    if (st != LA_OK) return st;
    const void *in[2] = {q, k};
    void *out[2] = {q_out, k_out};
    for (int i = 0; i < 2; ++i) {
        Side &s = p.side[i];
        if (s.H == 0 || B == 0 || N == 0) continue;
        s.x = in[i];
        s.y = out[i];
        s.sx = strides ? strides[i] : contiguous(s.H, N, d);
        s.sy = strides ? strides[2 + i] : contiguous(s.H, N, d);
        if (!s.x || !s.y) return qk_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
        if (negative(s.sx) || negative(s.sy))
            return qk_fail(LA_ERR_INVALID_ARG, who, "negative stride");
        if (!rows_disjoint(s.sy, B, s.H, N, d))
            return qk_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
        if (s.y == s.x && !same(s.sx, s.sy))
            return qk_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
    }
    if (B == 0 || N == 0 || Hq + Hk == 0) return LA_OK;
    if (Hq && Hk && (q_out == k || k_out == q || q_out == k_out))
        return qk_fail(LA_ERR_INVALID_ARG, who, "an output aliases the other side");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == LA_F32 ? launch<float, false>(who, p, s)
                           : launch<__nv_bfloat16, false>(who, p, s);
}

__attribute__((visibility("default")))
la_status la_backward_qk_norm_rope(const void *dq_out, const void *dk_out, const void *q,
                                   const void *k, void *dq, void *dk, float *dq_weight,
                                   float *dk_weight, const la_strides *strides,
                                   const void *q_weight, const void *k_weight, int norm,
                                   float eps, const la_rope *rope, int B, int Hq, int Hk, int N,
                                   int d, la_dtype dtype, la_dtype weight_dtype,
                                   la_stream_t stream) {
    const char *who = "la_backward_qk_norm_rope";
    Params p;
    la_status st = qk_common(who, p, q_weight, k_weight, norm, eps, rope, B, Hq, Hk, N, d, dtype,
                             weight_dtype);
    if (st != LA_OK) return st;
    if (!norm && (dq_weight || dk_weight))
        return qk_fail(LA_ERR_INVALID_ARG, who, "weight gradients need norm");
    if (dq_weight && dq_weight == dk_weight)
        return qk_fail(LA_ERR_INVALID_ARG, who, "one buffer for both weight gradients");
    const void *gin[2] = {dq_out, dk_out}, *xin[2] = {q, k};
    void *out[2] = {dq, dk};
    float *dw[2] = {dq_weight, dk_weight};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int i = 0; i < 2; ++i) {
        Side &sd = p.side[i];
        if (sd.H == 0 || B == 0 || N == 0) continue;
        sd.dy = gin[i];
        sd.x = norm ? xin[i] : nullptr;
        sd.y = out[i];
        sd.sdy = strides ? strides[i] : contiguous(sd.H, N, d);
        sd.sx = norm ? (strides ? strides[2 + i] : contiguous(sd.H, N, d)) : la_strides{0, 0, 0};
        sd.sy = strides ? strides[4 + i] : contiguous(sd.H, N, d);
        sd.dw = dw[i];
        if (!sd.dy || !sd.y || (norm && !sd.x))
            return qk_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
        if (negative(sd.sx) || negative(sd.sy) || negative(sd.sdy))
            return qk_fail(LA_ERR_INVALID_ARG, who, "negative stride");
        if (!rows_disjoint(sd.sy, B, sd.H, N, d))
            return qk_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
        if (sd.y == sd.dy && !same(sd.sdy, sd.sy))
            return qk_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
        if (norm && (sd.y == xin[0] || sd.y == xin[1]))
            return qk_fail(LA_ERR_INVALID_ARG, who, "an output aliases an input");
    }
    if (B && N && Hq && Hk && (dq == dk_out || dk == dq_out || dq == dk))
        return qk_fail(LA_ERR_INVALID_ARG, who, "an output aliases the other side");
    // a side without rows has a zero weight gradient
    for (int i = 0; i < 2; ++i)
        if (dw[i] && !p.side[i].dw) {
            const cudaError_t e = cudaMemsetAsync(dw[i], 0, sizeof(float) * d, s);
            if (e != cudaSuccess) return qk_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
        }
    if (B == 0 || N == 0 || Hq + Hk == 0) return LA_OK;
    return dtype == LA_F32 ? launch<float, true>(who, p, s)
                           : launch<__nv_bfloat16, true>(who, p, s);
}

}  // extern "C"

// What the operators of a layer around the attention share: vectors of values, the
// position rotation's angles, refusals and the checks of strides.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "la_internal.h"

namespace la {

// V values of T as they lie in memory: one load or store of V * sizeof(T) bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float &d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float x) { d = __float2bfloat16_rn(x); }

// bf16 pairs are taken apart and put together as 32-bit words: one instruction
// a value, and one a pair.
template <typename T, int V>
__device__ __forceinline__ void widen(const Pack<T, V> *p, float *e) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        struct alignas(2 * V) Words {
            unsigned u[V / 2];
        };
        const Words w = *reinterpret_cast<const Words *>(p);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            e[2 * i] = __uint_as_float(w.u[i] << 16);
            e[2 * i + 1] = __uint_as_float(w.u[i] & 0xffff0000u);
        }
    } else {
        const Pack<T, V> a = *p;
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = to_f(a.v[i]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void narrow(T *dst, const float *e) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        struct alignas(2 * V) Words {
            unsigned u[V / 2];
        } w;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 pair = __floats2bfloat162_rn(e[2 * i], e[2 * i + 1]);
            w.u[i] = reinterpret_cast<const unsigned &>(pair);
        }
        *reinterpret_cast<Words *>(dst) = w;
    } else {
        Pack<T, V> a;
#pragma unroll
        for (int i = 0; i < V; ++i) from_f(a.v[i], e[i]);
        *reinterpret_cast<Pack<T, V> *>(dst) = a;
    }
}

// cos and sin of pos * turns (2^-64 turns).  The top 32 bits are the angle in 2^-32
// turns.  For bf16 results the special function unit is exact enough: within [-pi,
// pi] it is off by 2^-21 at most, 2^-12 of half a step of the result.  Elsewhere (fp32
// rows, and backward, whose weight gradients are fp32) the angle is taken apart into
// quarter turns and a rest z of at most half a quarter, exactly, so that rounding the
// rest to fp32 costs 0.4 u (u = 2^-24; of the whole angle 1.6 u).  sin(pi/4 z) = z (s0
// + w S(w)) and cos(pi/4 z) = 1 + w C(w), w = z^2; S and C interpolate the exact
// quotients at the Chebyshev nodes of [0, 1], off by 0.2 u at most, s0 is pi/4 as two
// fp32 numbers.  Each result is within 1.4 u.
template <bool kFine>
__device__ __forceinline__ void turn_of(long long pos, unsigned long long turns, float *c,
                                        float *s) {
    const unsigned t = (unsigned)(((unsigned long long)pos * turns) >> 32);
    if (!kFine) {
        __sincosf((float)(int)t * 1.46291807926715968e-9f, s, c);  // pi 2^-31
        return;
    }
    const unsigned quarter = (t + 0x20000000u) >> 30;
    const float z = (float)(int)(t - (quarter << 30)) * 0x1p-29f, w = z * z;
    float a = fmaf(w, -3.61091152e-5f, 2.49021966e-3f);
    a = fmaf(w, a, -8.07455033e-2f);
    a = fmaf(w, a, -2.18556941e-8f);
    a = fmaf(z, 0.785398185f, z * a);
    float b = fmaf(w, 3.54195276e-6f, -3.25961388e-4f);
    b = fmaf(w, b, 1.58543382e-2f);
    b = fmaf(w, b, -0.308425128f);
    b = fmaf(w, b, 1.f);
    const float sine = quarter & 1 ? b : a, cosine = quarter & 1 ? a : b;
    *s = quarter & 2 ? -sine : sine;
    *c = (quarter + 1) & 2 ? -cosine : cosine;
}

// Whether no two rows of d elements overlap.
inline bool rows_disjoint(const la_strides &s, int B, int H, int N, int d) {
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

// f / (2 pi) mod 1 in 2^-64 turns, |f| <= 1e9.  1 / (2 pi) is the sum of two
// doubles, so the product is good to about 2^-64 turns for |f| up to a few turns.
inline unsigned long long turns_of(double f) {
    if (f < 0) return 0 - turns_of(-f);
    const double c = 0.15915494309189535, c_low = -9.839338337591243e-18;
    const double t = f * c;
    const double low = std::fma(f, c, -t) + f * c_low;  // |low| < 2^-51 |t| < 2^-23
    const double part = t - std::floor(t);              // exact, in [0, 1)
    // a double below 1 is a whole number of 2^-64 from 2^-11 on, and loses less
    // than one below
    return (unsigned long long)(part * 0x1p64) + (unsigned long long)(long long)(low * 0x1p64);
}

inline la_status layer_fail(la_status s, const char *who, const char *msg) {
    char text[200];
    std::snprintf(text, sizeof(text), "%s: %s", who, msg);
    set_last_error(text);
    return s;
}

inline la_strides contiguous(int H, int N, int d) {
    return {(long long)H * N * d, (long long)N * d, d};
}

inline bool negative(const la_strides &s) { return s.b < 0 || s.h < 0 || s.n < 0; }

// a i / n, in 32 bits where that is enough.
__device__ __forceinline__ long long share_of(long long a, int i, int n) {
    const long long x = a * i;
    return x <= 0xffffffffLL ? (long long)((unsigned)x / (unsigned)n) : x / n;
}

// Equal pieces of a list of work whose length only the device knows: for each of B
// entries, `segs` stretches of tiles_of(b) > 0 tiles.  A block's piece is [x0, x1) of
// `total` tiles, and x0 is tile `rest` of entry b's stretches.  There are `pieces` of
// them, at most one for each block and of `least` tiles or more where the list is that
// long, so that no piece between others is empty; later blocks have x0 == x1.
struct Piece {
    long long total, x0, x1, rest;
    int pieces, b;

    // The piece that holds tile x.
    __device__ __forceinline__ int of(long long x) const {
        return (int)(((x + 1) * pieces - 1) / total);
    }
};

// The same where every entry has `tiles` tiles a stretch.
__device__ __forceinline__ Piece even_piece(int B, int segs, int least, int tiles) {
    Piece p;
    p.total = (long long)B * segs * tiles;
    p.pieces = (int)min((long long)gridDim.x, max(1LL, share_of(p.total, 1, least)));
    p.x0 = share_of(p.total, min((int)blockIdx.x, p.pieces), p.pieces);
    p.x1 = share_of(p.total, min((int)blockIdx.x + 1, p.pieces), p.pieces);
    const long long per = (long long)segs * tiles;
    p.b = (int)(p.x0 <= 0x7fffffff && per <= 0x7fffffff ? (unsigned)p.x0 / (unsigned)per
                                                         : p.x0 / per);
    p.rest = p.x0 - p.b * per;
    return p;
}

// All kThreads threads of a block call this; `shared` has kThreads / 32 + 2 numbers.
template <int kThreads, typename F>
__device__ __forceinline__ Piece find_piece(int B, int segs, int least, F tiles_of,
                                            long long *shared) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += tiles_of(b);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long other = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += other;
    }
    if (lane == 31) shared[warp] = upto;
    __syncthreads();
    Piece p;
    long long base = 0;
    p.total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += shared[w];
        p.total += shared[w];
    }
    p.total *= segs;
    p.pieces = (int)min((long long)gridDim.x, max(1LL, share_of(p.total, 1, least)));
    p.x0 = share_of(p.total, min((int)blockIdx.x, p.pieces), p.pieces);
    p.x1 = share_of(p.total, min((int)blockIdx.x + 1, p.pieces), p.pieces);
    long long at = (base + upto - mine) * segs;  // of this thread's first entry
    if (p.x0 >= at && p.x0 < at + mine * segs) {
        int b = b0;
        for (;; ++b) {
            const long long n = (long long)tiles_of(b) * segs;
            if (p.x0 < at + n) break;
            at += n;
        }
        shared[kWarps] = b;
        shared[kWarps + 1] = p.x0 - at;
    }
    __syncthreads();
    p.b = (int)shared[kWarps];
    p.rest = shared[kWarps + 1];
    return p;
}

// The checks of a paged cache that every call of one makes.
inline la_status check_cache(const char *who, const la_cache *c, int B, int Hk, int d,
                             la_dtype dtype) {
    if (B < 0 || Hk < 0) return layer_fail(LA_ERR_INVALID_ARG, who, "negative B or Hk");
    if (d < 1 || d > LA_MAX_D) return layer_fail(LA_ERR_INVALID_ARG, who, "d must be in 1..256");
    if (dtype != LA_F32 && dtype != LA_BF16)
        return layer_fail(LA_ERR_INVALID_ARG, who, "unknown dtype");
    if (!c) return layer_fail(LA_ERR_INVALID_ARG, who, "null cache");
    if (c->pages < 0 || c->max_pages < 0)
        return layer_fail(LA_ERR_INVALID_ARG, who, "negative pages or max_pages");
    if (c->page_size < 1) return layer_fail(LA_ERR_INVALID_ARG, who, "page_size must be positive");
    if ((long long)c->max_pages * c->page_size > 1 << 30)
        return layer_fail(LA_ERR_UNSUPPORTED, who, "the table holds more than 2^30 tokens");
    if (c->table_stride < 0 || negative(c->k_strides) || negative(c->v_strides))
        return layer_fail(LA_ERR_INVALID_ARG, who, "negative stride");
    if (B == 0) return LA_OK;
    if (!c->lengths || (c->max_pages && !c->table))
        return layer_fail(LA_ERR_INVALID_ARG, who, "null table or lengths");
    if ((uintptr_t)c->lengths % 4 || (uintptr_t)c->table % 4)
        return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned table or lengths");
    if (Hk == 0 || c->pages == 0) return LA_OK;
    const uintptr_t elem = dtype == LA_F32 ? 4 : 2;
    if (!c->k || !c->v) return layer_fail(LA_ERR_INVALID_ARG, who, "null cache pointer");
    if ((uintptr_t)c->k % elem || (uintptr_t)c->v % elem)
        return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned cache pointer");
    if (c->k == c->v) return layer_fail(LA_ERR_INVALID_ARG, who, "one buffer for keys and values");
    return LA_OK;
}

}  // namespace la

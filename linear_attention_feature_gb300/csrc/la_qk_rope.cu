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
//
// What bounds it (GB300, 6.78 TB/s measured copy): memory, once the angles are
// shared by a token's heads, rows arrive asynchronously and the arithmetic goes
// through the packed fp32 instructions.  Forward 2 x (16 + 16) x 32768 x 128 bf16,
// token-major to head-major: 182 us, 5.9 TB/s (13 instructions a value); 4 x (16 +
// 16) x 4096 x 64: 21 us, 6.4 TB/s.  Backward 4 x (8 + 8) x 16384 x 128: 135 us, 6.0
// TB/s (25 instructions a value, the weights' sums among them).  First kernel,
// one warp per row: 1332, 233 and 1021 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "la_internal.h"
#include "la_layer.cuh"
#include "la_tc.h"
#include "la_tc_host.h"
#include "la_tc_ptx.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = LA_MAX_D / 2;

// One side (queries or keys) of a call.  Strides are in elements.
struct Side {
    const void *x;   // forward input
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
    int sums_at;     // and where the threads' sums lie in shared memory
    // the split of the work, see qk_rows_kernel
    int lane_bits, token_bits, blocks_q;
    unsigned long long turns[kMaxPairs];  // frequency, 2^-64 turns per position
};

// V values to shared memory, asynchronously (4 bytes or more).  The input is read
// once: it leaves L2 first (the 2 x 16 x 32768 x 128 call 190 -> 182 us).
template <typename T, int V>
__device__ __forceinline__ void fetch(Pack<T, V> *dst, const T *src, uint64_t policy) {
    constexpr int kBytes = (int)sizeof(T) * V;
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(d),
                     "l"(src), "l"(policy) : "memory");
    else
        asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %2, %3;" ::"r"(d),
                     "l"(src), "n"(kBytes < 4 ? 4 : kBytes), "l"(policy) : "memory");
}

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

// Sum over a row of K S chunks of 2 P / S terms in each of 2^bits lanes, N sums
// at once.  Term e of chunk c in lane l stands for pair ((c << bits) + l) 2 P / S +
// e; the sum is the binary tree over the pair's bits from the lowest up, so that
// it does not depend on the vectors: a row gives the same bits whatever its
// alignment.
template <int S, int N, int K, int P>
__device__ __forceinline__ void row_sum(float2 (&t)[N][K][P], int bits, float (&sum)[N]) {
    constexpr int C = K * S;
    float u[N][C];
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float w[2 * P];
#pragma unroll
            for (int e = 0; e < P; ++e) w[2 * e] = t[q][j][e].x, w[2 * e + 1] = t[q][j][e].y;
#pragma unroll
            for (int o = 1; o < 2 * P / S; o *= 2)
#pragma unroll
                for (int e = 0; e < 2 * P; e += 2 * o) w[e] = __fadd_rn(w[e], w[e + o]);
#pragma unroll
            for (int c = 0; c < S; ++c) u[q][j * S + c] = w[c * (2 * P / S)];
        }
    for (int o = 1; o >> bits == 0; o <<= 1)
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
            for (int j = 0; j < C; ++j) u[q][j] += __shfl_xor_sync(~0u, u[q][j], o);
#pragma unroll
    for (int q = 0; q < N; ++q) {
#pragma unroll
        for (int o = 1; o < C; o *= 2)
#pragma unroll
            for (int j = 0; j < C; j += 2 * o) u[q][j] += u[q][j + o];
        sum[q] = u[q][0];
    }
}

// a becomes the rounded a + x and x what the rounding left out, exactly.  (Where the
// sum is not finite, x is left at some finite value: a minimum drops the NaN.)
__device__ __forceinline__ void two_sum(float &a, float &x) {
    const float s = __fadd_rn(a, x), b = __fsub_rn(s, a);
    x = fminf(__fadd_rn(__fsub_rn(a, __fsub_rn(s, b)), __fsub_rn(x, b)), 1e30f);
    a = s;
}

// The same in three operations, exactly where |x| <= |a|, else within u |x|.
__device__ __forceinline__ void quick_two_sum(float &a, float &x) {
    const float s = __fadd_rn(a, x);
    x = fminf(__fsub_rn(x, __fsub_rn(s, a)), 1e30f);
    a = s;
}

// Rows that a thread adds to its sums of g n before they go to its larger sums.
constexpr int kFold = 16;
// Rows in flight per thread.
template <bool kBack>
constexpr int ring_depth() { return kBack ? 3 : 4; }
// Single bf16 values cannot be copied asynchronously: the lanes of a row copy the
// 16-byte units of memory that hold it, wherever it begins in the first of them.
template <typename T, int V>
constexpr bool whole_rows() { return sizeof(T) * V < 4; }
// Vectors of one of a lane's K parts of a row.
template <int V>
constexpr int vectors() { return V == 1 ? 4 : 2; }
// Bytes that a row's units take.
__host__ __device__ inline int row_units(int d) { return (2 * d + 14 + 15) / 16 * 16; }
template <typename T, int V, int K, bool kBack>
int ring_bytes(int d, int lane_bits) {
    return ring_depth<kBack>() * (kBack ? 2 : 1) *
           (whole_rows<T, V>() ? (kThreads >> lane_bits) * row_units(d)
                               : K * vectors<V>() * kThreads * V * (int)sizeof(T));
}
// Bytes of the threads' larger sums, behind the ring.
template <int V, int K>
constexpr int sums_bytes() { return kThreads * K * ((V + 1) / 2) * 2 * (int)sizeof(float2); }

// A row is shared by 2^lane_bits lanes of a warp.  A lane takes K parts of V
// pairs, each as two vectors of V values, such that both values of a pair are in
// one thread and a warp's access covers memory without gaps: where pairs are
// neighbours (kInter), the vectors of V / 2 pairs of two chunks 2^lane_bits
// vectors apart (vectors side by side in a lane leave half of each 32 bytes to the
// next access: 2 x (16 + 16) x 8192 x 128 fp32 127 us, 92 us with them apart); else
// the features i and i + half in the rotated part, i + half and i + d / 2 in the
// rest.  With V = 1 a part is two pairs of two chunks, four single values; an odd
// d leaves the last alone and makes the unrotated pairs neighbours.
//
// A block keeps to one side.  Its groups of lanes are a tile of 2^token_bits
// tokens times as many heads as are left, so a tile is H / heads rows per group;
// the rows of all tiles form one list, of which every block takes an equal piece.
// Angles are formed once per token and lane and serve the tile's rows.  Rows
// travel through a ring in shared memory, filled by cp.async some rows ahead;
// every thread reads only what it copied itself, so the ring needs no barrier
// (with whole_rows, what its row's lanes copied: a warp barrier).
//
// Backward, the sums of g n are in registers for kFold rows, then added to sums in
// shared memory.  What that addition rounds off stays behind in the registers, so
// the number of rows does not add to the error: dw is off by at most 19 u sum |g n|
// (u = 2^-24: 8.5 for chains of 16 rows, 5 for the lanes, one each for a chain's
// residue, a thread's sum, a block's, the last and the products).  One chain over
// all rows of a thread was off by several times as much and grew with them.
template <typename T, int V, int K, bool kInter, bool kBack>
__global__ void __launch_bounds__(kThreads, 2) qk_rows_kernel(const __grid_constant__ Params p) {
    constexpr int P = (V + 1) / 2;  // packed pairs per part
    constexpr int kVecs = vectors<V>();
    constexpr int kChunks = kInter || V == 1 ? 2 : 1;  // per part
    constexpr int kDepth = ring_depth<kBack>(), kSrc = kBack ? 2 : 1;
    constexpr bool kWhole = whole_rows<T, V>();
    extern __shared__ __align__(16) char smem[];
    __shared__ unsigned long long turns[kMaxPairs];
    __shared__ __align__(32) float weight[LA_MAX_D];
    Pack<T, V> *ring = reinterpret_cast<Pack<T, V> *>(smem) + threadIdx.x;

    const int bits = p.lane_bits, lane = threadIdx.x & ((1 << bits) - 1);
    const int group = threadIdx.x >> bits;
    const int tok_in = group & ((1 << p.token_bits) - 1), head_in = group >> p.token_bits;
    const int head_step = (kThreads >> bits) >> p.token_bits;
    const int pairs = (p.d + 1) / 2;
    const long long tokens = (long long)p.B * p.N;

    const int which = (int)blockIdx.x >= p.blocks_q;
    const Side sd = which ? p.side[1] : p.side[0];
    const int H = sd.H, rows = (H + head_step - 1) / head_step;  // per tile
    const long long total = ((tokens + (1 << p.token_bits) - 1) >> p.token_bits) * rows;
    const int blocks = which ? gridDim.x - p.blocks_q : p.blocks_q;
    const int block = which ? blockIdx.x - p.blocks_q : blockIdx.x;
    const long long it0 = total * block / blocks;
    const int count = (int)(total * (block + 1) / blocks - it0);  // rows of this block's groups

    if (kBack) tc::grid_dep_launch();
    for (int i = threadIdx.x; i < p.half; i += kThreads) turns[i] = p.turns[i];
    for (int i = threadIdx.x; i < p.d; i += kThreads) weight[i] = weight_at(sd.w, p.w_bf16, i);
    __syncthreads();

    auto pair = [&](int j, int e) {  // pair e < 2 P of part j
        constexpr int n = 2 * P / kChunks;  // per chunk
        return (lane + ((j * kChunks + e / n) << bits)) * n + e % n;
    };
    int at[K][kVecs];  // the vectors' first features
    bool has[K][kVecs];
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int m = 0; m < kVecs; ++m) {
            const int i = pair(j, V == 1 ? m / 2 : kInter ? m * P : 0);
            const bool rot = i < p.half, next = kInter || (!rot && p.d % 2);
            if (kInter && V > 1)
                at[j][m] = 2 * i;
            else if (m % 2 == 0)
                at[j][m] = next ? 2 * i : rot ? i : i + p.half;
            else
                at[j][m] = next ? 2 * i + 1 : rot ? i + p.half : i + p.d / 2;
            has[j][m] = i < pairs && at[j][m] < p.d;
        }

    // the batch entry and token of this group in a tile
    auto locate = [&](long long tile, int &b, int &n) {
        const long long tok = (tile << p.token_bits) + tok_in;
        const bool ok = tok < tokens;
        b = !ok ? 0 : tokens <= 0x7fffffff ? (int)((unsigned)tok / (unsigned)p.N) : (int)(tok / p.N);
        n = ok ? (int)(tok - (long long)b * p.N) : 0;
        return ok;
    };
    auto slot = [&](int depth, int src, int j, int m) {
        return ring + (((depth * kSrc + src) * K + j) * kVecs + m) * kThreads;
    };

    auto row_slot = [&](int depth, int src) {  // with kWhole
        return smem + ((depth * kSrc + src) * (kThreads >> bits) + group) * row_units(p.d);
    };
    auto fetch_units = [&](char *dst, const T *src) {
        const uintptr_t at = (uintptr_t)src, from = at & ~(uintptr_t)15;
        const int end = (int)(at & 15) + p.d * (int)sizeof(T);
        for (int u = 16 * lane; u < end; u += 16 << bits)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             (unsigned)__cvta_generic_to_shared(dst + u)), "l"(from + u) : "memory");
    };

    // the copying side of the ring
    const uint64_t policy = tc::policy_evict_first();
    long long f_tile = it0 / rows;
    int f_left = count, f_row = (int)(it0 - f_tile * rows), f_depth = 0;
    bool f_ok = false;
    const T *fx = nullptr, *fg = nullptr;  // the next row
    const long long fx_step = head_step * sd.sx.h, fg_step = head_step * sd.sdy.h;
    auto f_enter = [&]() {
        int b, n;
        f_ok = locate(f_tile, b, n);
        const int h = head_in + f_row * head_step;
        fx = static_cast<const T *>(sd.x) + b * sd.sx.b + n * sd.sx.n + h * sd.sx.h;
        if (kBack) fg = static_cast<const T *>(sd.dy) + b * sd.sdy.b + n * sd.sdy.n + h * sd.sdy.h;
    };
    f_enter();
    auto fetch_row = [&]() {
        if (f_left > 0) {
            const bool ok = f_ok && head_in + f_row * head_step < H;
            if (kWhole && ok) {
                fetch_units(row_slot(f_depth, 0), fx);
                if (kBack) fetch_units(row_slot(f_depth, kSrc - 1), fg);
            }
#pragma unroll
            for (int j = 0; j < K && !kWhole; ++j)
#pragma unroll
                for (int m = 0; m < kVecs; ++m) {
                    if (!ok || !has[j][m]) continue;
                    fetch<T, V>(slot(f_depth, 0, j, m), fx + at[j][m], policy);
                    if (kBack) fetch<T, V>(slot(f_depth, kSrc - 1, j, m), fg + at[j][m], policy);
                }
            f_depth = f_depth + 1 == kDepth ? 0 : f_depth + 1;
            --f_left;
            fx += fx_step;
            fg += fg_step;
            if (++f_row == rows) {
                f_row = 0;
                ++f_tile;
                f_enter();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (!kWhole)  // lanes and rows without values read zeros, or what an earlier row left
#pragma unroll
        for (int i = 0; i < kDepth * kSrc * K * kVecs; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) ring[i * kThreads].v[e] = T(0.f);
    for (int i = 0; i < kDepth - 1; ++i) fetch_row();

    // the values of a part's vectors as the pairs' first and second ones, and
    // where value i of those lies
    auto sort = [&](const float (&e)[4 * P], float2 (&m0)[P], float2 (&m1)[P]) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (kChunks == 2) {
                m0[i] = make_float2(e[4 * i], e[4 * i + 2]);
                m1[i] = make_float2(e[4 * i + 1], e[4 * i + 3]);
            } else {
                m0[i] = make_float2(e[2 * i], e[2 * i + 1]);
                m1[i] = make_float2(e[2 * P + 2 * i], e[2 * P + 2 * i + 1]);
            }
        }
    };
    auto place = [](int second, int i) {
        return kChunks == 2 ? 2 * i + second : second * 2 * P + i;
    };
    // part j of source src in a place of the ring; `begin` is the row's address
    // where whole rows are copied
    auto open = [&](int depth, int src, int j, bool ok, unsigned begin, float2 (&m0)[P],
                    float2 (&m1)[P]) {
        float e[4 * P];
#pragma unroll
        for (int m = 0; m < kVecs; ++m)
            if constexpr (kWhole) {
                const T *r = reinterpret_cast<const T *>(row_slot(depth, src) + (begin & 15u));
                e[m] = ok && has[j][m] ? to_f(r[at[j][m]]) : 0.f;
            } else {
                widen(slot(depth, src, j, m), e + m * V);
            }
        sort(e, m0, m1);
    };

    // Backward with the longest vectors the weights are read again for each row: in
    // registers they made the kernel spill (4 x (8 + 8) x 16384 x 128: 149 us, 135 us
    // read again; shorter vectors have the registers).
    constexpr bool kReread = kBack && V == 8;
    float2 w0[K][P], w1[K][P], dw0[K][P], dw1[K][P];
    auto weigh = [&](int j) {
        float e[4 * P];
        if constexpr (kReread) {
#pragma unroll
            for (int m = 0; m < kVecs; ++m) {
                Pack<float, V> w = {};
                if (has[j][m]) w = *reinterpret_cast<const Pack<float, V> *>(weight + at[j][m]);
#pragma unroll
                for (int i = 0; i < V; ++i) e[m * V + i] = w.v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4 * P; ++i)
                e[i] = has[j][i / V] ? weight[at[j][i / V] + i % V] : 0.f;
        }
        sort(e, w0[j], w1[j]);
    };
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (!kReread) weigh(j);
#pragma unroll
        for (int i = 0; i < P; ++i) dw0[j][i] = dw1[j][i] = make_float2(0.f, 0.f);
    }
    const bool summing = kBack && p.partial;
    float2 *const sums = reinterpret_cast<float2 *>(smem + p.sums_at) + threadIdx.x;
    if (summing)
        for (int i = 0; i < 2 * K * P; ++i) sums[i * kThreads] = make_float2(0.f, 0.f);
    auto fold = [&]() {
#pragma unroll
        for (int i = 0; i < 2 * K * P; ++i) {
            float2 &x = (i % 2 ? dw1 : dw0)[i / 2 / P][i / 2 % P], a = sums[i * kThreads];
            quick_two_sum(a.x, x.x);
            quick_two_sum(a.y, x.y);
            sums[i * kThreads] = a;
        }
    };

    // Features beyond the rotated ones pass as they are: a cosine of 1 and a sine of 0
    // would make a NaN of one beside a value that is not finite.  With halves as pairs
    // a lane's part of long vectors is rotated or passes as a whole; elsewhere each
    // pair is looked at, where any pass (backward 4 x (8 + 8) x 16384 x 128: 152 us with
    // half of the features rotated, as neighbours, 146 with all; a branch around each
    // chunk of neighbouring pairs was 1 % faster with half of them, 9 % slower with all).
    constexpr bool kWholeParts = V >= 4 && !kInter;
    const bool some_pass = p.half < pairs;
    auto passes = [&](int j, int e) { return pair(j, e) >= p.half; };

    int depth = 0;
    long long tile = it0 / rows;
    int row = (int)(it0 - tile * rows);
    const long long y_step = head_step * sd.sy.h;
    for (int left = count; left > 0;) {
        int b, n;
        const bool t_ok = locate(tile, b, n);
        T *y = static_cast<T *>(sd.y) + b * sd.sy.b + n * sd.sy.n +
               (head_in + row * head_step) * sd.sy.h;
        const long long pos = p.half && t_ok ? position_of(p, b, n) : 0;
        float2 cs[K][P], sn[K][P];
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < 2 * P; ++e) {
                const int i = pair(j, e);
                float c = 1.f, s = 0.f;
                if (i < p.half) turn_of<sizeof(T) == 4 || kBack>(pos, turns[i], &c, &s);
                (e % 2 ? cs[j][e / 2].y : cs[j][e / 2].x) = c;
                (e % 2 ? sn[j][e / 2].y : sn[j][e / 2].x) = s;
            }
        unsigned at_x = 0, at_g = 0;  // addresses of the rows, with kWhole
        if (kWhole) {
            const long long h = head_in + row * head_step;
            at_x = (unsigned)((uintptr_t)sd.x +
                              (b * sd.sx.b + n * sd.sx.n + h * sd.sx.h) * sizeof(T));
            at_g = (unsigned)((uintptr_t)sd.dy +
                              (b * sd.sdy.b + n * sd.sdy.n + h * sd.sdy.h) * sizeof(T));
        }
        for (; row < rows && left > 0; ++row, --left, y += y_step) {
            if (kWhole) __syncwarp();  // the place that is filled next has been read
            fetch_row();
            if (summing && left % kFold == 0) fold();
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            if (kWhole) __syncwarp();
            const bool ok = t_ok && head_in + row * head_step < H;

            float2 v0[K][P], v1[K][P], g0[K][P], g1[K][P], t[kSrc][K][P];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                open(depth, 0, j, ok, at_x, v0[j], v1[j]);
                if (kBack) open(depth, kSrc - 1, j, ok, at_g, g0[j], g1[j]);
                if (kReread) weigh(j);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    t[0][j][i] = __ffma2_rn(v0[j][i], v0[j][i], __fmul2_rn(v1[j][i], v1[j][i]));
                if (!kBack) continue;
                // turned back; what the sine multiplies is 0 where a pair passes
                float2 ga[P], gc[P];
#pragma unroll
                for (int i = 0; i < P; ++i) ga[i] = g0[j][i], gc[i] = g1[j][i];
                if (!kWholeParts && some_pass)
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        if (passes(j, 2 * i)) ga[i].x = gc[i].x = 0.f;
                        if (passes(j, 2 * i + 1)) ga[i].y = gc[i].y = 0.f;
                    }
                if (!kWholeParts || !passes(j, 0))
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const float2 a = g0[j][i], c = g1[j][i], as = __fmul2_rn(ga[i], sn[j][i]);
                        g0[j][i] = __ffma2_rn(a, cs[j][i], __fmul2_rn(gc[i], sn[j][i]));
                        g1[j][i] = make_float2(fmaf(c.x, cs[j][i].x, -as.x),
                                               fmaf(c.y, cs[j][i].y, -as.y));
                    }
                // then times the weight for dx
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    t[kSrc - 1][j][i] =
                        __ffma2_rn(v0[j][i], __fmul2_rn(w0[j][i], g0[j][i]),
                                   __fmul2_rn(v1[j][i], __fmul2_rn(w1[j][i], g1[j][i])));
                }
            }
            float r = 1.f, m = 0.f;
            if (kBack || p.norm) {
                float sum[kSrc];
                row_sum<kChunks>(t, bits, sum);
                r = rsqrtf(fmaf(sum[0], p.inv_d, p.eps));
                // n w g summed is r sum(v w g)
                if (kBack) m = __fmul_rn(__fmul_rn(sum[kSrc - 1], p.inv_d), r);
            }
            const float2 r2 = make_float2(r, r), m2 = make_float2(-m, -m);
            float2 o0[K][P], o1[K][P];
#pragma unroll
            for (int j = 0; j < K; ++j)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 n0 = __fmul2_rn(v0[j][i], r2), n1 = __fmul2_rn(v1[j][i], r2);
                    if (!kBack) {
                        const float2 a = __fmul2_rn(n0, w0[j][i]), c = __fmul2_rn(n1, w1[j][i]);
                        o0[j][i] = a;
                        o1[j][i] = c;
                        if (!kWholeParts || !passes(j, 0)) {
                            const float2 cn = __fmul2_rn(c, sn[j][i]);
                            o0[j][i] = make_float2(fmaf(a.x, cs[j][i].x, -cn.x),
                                                fmaf(a.y, cs[j][i].y, -cn.y));
                            o1[j][i] = __ffma2_rn(c, cs[j][i], __fmul2_rn(a, sn[j][i]));
                        }
                    } else {
                        if (ok) {  // other rows hold what an earlier one left
                            dw0[j][i] = __ffma2_rn(g0[j][i], n0, dw0[j][i]);
                            dw1[j][i] = __ffma2_rn(g1[j][i], n1, dw1[j][i]);
                        }
                        o0[j][i] = __fmul2_rn(
                            r2, __ffma2_rn(n0, m2, __fmul2_rn(w0[j][i], g0[j][i])));
                        o1[j][i] = __fmul2_rn(
                            r2, __ffma2_rn(n1, m2, __fmul2_rn(w1[j][i], g1[j][i])));
                    }
                }
            if (!kBack && !kWholeParts && some_pass)
#pragma unroll
                for (int j = 0; j < K; ++j)
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const float2 a = __fmul2_rn(__fmul2_rn(v0[j][i], r2), w0[j][i]);
                        const float2 c = __fmul2_rn(__fmul2_rn(v1[j][i], r2), w1[j][i]);
                        if (passes(j, 2 * i)) o0[j][i].x = a.x, o1[j][i].x = c.x;
                        if (passes(j, 2 * i + 1)) o0[j][i].y = a.y, o1[j][i].y = c.y;
                    }
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float e[4 * P];
#pragma unroll
                for (int i = 0; i < 2 * P; ++i) {
                    e[place(0, i)] = i % 2 ? o0[j][i / 2].y : o0[j][i / 2].x;
                    e[place(1, i)] = i % 2 ? o1[j][i / 2].y : o1[j][i / 2].x;
                }
#pragma unroll
                for (int m = 0; m < kVecs; ++m)
                    if (ok && has[j][m]) narrow<T, V>(y + at[j][m], e + m * V);
            }
            depth = depth + 1 == kDepth ? 0 : depth + 1;
            at_x += (unsigned)(fx_step * sizeof(T));
            at_g += (unsigned)(fg_step * sizeof(T));
        }
        row = 0;
        ++tile;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    if (!summing) return;
    // the block's sums: over the groups of each warp, then over the warps, in
    // the ring's memory
    fold();
#pragma unroll
    for (int i = 0; i < 2 * K * P; ++i)
        (i % 2 ? dw1 : dw0)[i / 2 / P][i / 2 % P] = sums[i * kThreads];
    __syncthreads();
    float(*sum)[LA_MAX_D] = reinterpret_cast<float(*)[LA_MAX_D]>(smem);
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) {
            float a = e % 2 ? dw0[j][e / 2].y : dw0[j][e / 2].x;
            float c = e % 2 ? dw1[j][e / 2].y : dw1[j][e / 2].x;
            for (int o = 1 << bits; o < 32; o <<= 1) {
                a += __shfl_xor_sync(~0u, a, o);
                c += __shfl_xor_sync(~0u, c, o);
            }
            const int i0 = place(0, e), i1 = place(1, e);
            if ((threadIdx.x & 31) == lane) {
                if (has[j][i0 / V]) sum[warp][at[j][i0 / V] + i0 % V] = a;
                if (has[j][i1 / V]) sum[warp][at[j][i1 / V] + i1 % V] = c;
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += kThreads) {
        float t = 0.f, low = 0.f;
        for (int q = 0; q < kThreads / 32; ++q) {
            float x = sum[q][i];
            two_sum(t, x);
            low += x;
        }
        p.partial[(long long)blockIdx.x * p.d + i] = t + low;
    }
}

// dw[i] = the sum of the blocks' partial sums, in order for each of 32 interleaved
// parts, then over the parts, every addition with what it rounds off kept in a second
// sum.  A block takes 32 features of one side.  A few microseconds of latency, most
// of them hidden by starting it while the rows' kernel ends.
__global__ void __launch_bounds__(1024)
qk_weight_kernel(const float *partial, int blocks_q, int blocks, int d, float *dwq, float *dwk) {
    // started while the rows' kernel runs: its sums are there after this
    tc::grid_dep_wait();
    const int chunks = (d + 31) / 32, side = (int)blockIdx.x >= chunks;
    float *dw = side ? dwk : dwq;
    if (!dw) return;
    __shared__ float2 sum[32][32];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int i = ((int)blockIdx.x - side * chunks) * 32 + lane;
    const int b0 = side ? blocks_q : 0, b1 = side ? blocks : blocks_q;
    float t = 0.f, low = 0.f;
    if (i < d)
#pragma unroll 8
        for (int b = b0 + part; b < b1; b += 32) {
            float x = partial[(long long)b * d + i];
            two_sum(t, x);
            low += x;
        }
    sum[part][lane] = make_float2(t, low);
    __syncthreads();
    if (part > 0 || i >= d) return;
    for (int q = 1; q < 32; ++q) {
        float2 x = sum[q][lane];
        two_sum(t, x.x);
        low += x.x + x.y;
    }
    dw[i] = t + low;
}

bool same(const la_strides &a, const la_strides &b) {
    return a.b == b.b && a.h == b.h && a.n == b.n;
}

// Values per access: the most (a power of two, up to `most`) that divide the row and
// its rotated part (where pairs are not neighbours, their halves) and at which every
// row of every tensor is aligned.
int vector_of(const Params &p, int most, int elem) {
    // a power of two divides all of these if it divides their union
    unsigned long long all =
        (unsigned)(p.interleaved ? p.d | 2 * p.half : p.half | (p.d % 2 ? 1 : p.d / 2)) | (unsigned)most;
    auto add = [&](const void *q, const la_strides &s, int H) {
        all |= (uintptr_t)q / (uintptr_t)elem;
        if (p.B > 1) all |= (unsigned long long)s.b;
        if (H > 1) all |= (unsigned long long)s.h;
        if (p.N > 1) all |= (unsigned long long)s.n;
    };
    for (const Side &s : p.side) {
        if (s.H == 0) continue;
        add(s.x, s.sx, s.H);
        add(s.dy, s.sdy, s.H);
        add(s.y, s.sy, s.H);
    }
    return (int)(all & (0 - all));
}

template <typename T, int V, int K, bool kBack>
cudaError_t launch_rows(Params &p, unsigned blocks, cudaStream_t stream) {
    auto kern = p.interleaved ? qk_rows_kernel<T, V, K, true, kBack>
                              : qk_rows_kernel<T, V, K, false, kBack>;
    // the sums of the weight gradient, 8 rows of LA_MAX_D, share the ring
    int smem = std::max(ring_bytes<T, V, K, kBack>(p.d, p.lane_bits),
                        kThreads / 32 * LA_MAX_D * 4);
    if (p.partial) {
        p.sums_at = smem;
        smem += sums_bytes<V, K>();
    }
    if (smem > 40 * 1024) {  // 48 KB with the static arrays need no attribute
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<blocks, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

// Blocks of one call at most: two run on an SM at once.
long long resident_blocks(int sms) { return 2LL * sms; }

template <typename T, bool kBack>
la_status launch(const char *who, Params &p, void *workspace, size_t workspace_bytes,
                 cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e != cudaSuccess) return layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    const int v = vector_of(p, 16 / (int)sizeof(T), (int)sizeof(T));
    const int chunks = ((p.d + 1) / 2 + v - 1) / v;  // of a row
    // Pairs / V per lane: more of the small ones, so that a warp takes more rows at a
    // time (2 x 24 x 4000 rows of 66 bf16 values: 60 us with two single pairs per
    // lane, 41 us with four; of 36: 20 us with one double pair, 14 us with two).
    const int per_lane = v >= 4 ? 1 : v == 2 ? 2 : 4;
    while (per_lane << p.lane_bits < chunks) ++p.lane_bits;
    const int groups = kThreads >> p.lane_bits;
    const long long tokens = (long long)p.B * p.N;
    while ((1 << p.token_bits) < groups && (1 << p.token_bits) < tokens) ++p.token_bits;
    const int head_step = groups >> p.token_bits;
    const long long tiles = (tokens + (1 << p.token_bits) - 1) >> p.token_bits;
    // as many blocks as run at once, shared by the sides as their rows
    const long long most = resident_blocks(sms);
    long long total[2];
    for (int i = 0; i < 2; ++i) total[i] = tiles * ((p.side[i].H + head_step - 1) / head_step);
    long long bq = total[0], bk = total[1];
    if (bq + bk > most) {
        const double share = (double)total[0] / (double)(total[0] + total[1]);
        bq = bq ? std::max(1LL, std::min(most - (bk ? 1 : 0), std::llround(share * most))) : 0;
        bk = bk ? most - bq : 0;
    }
    p.blocks_q = (int)bq;
    const long long blocks = bq + bk;
    void *ws = nullptr;
    const bool want_dw = kBack && (p.side[0].dw || p.side[1].dw);
    const size_t need = sizeof(float) * (size_t)blocks * p.d;
    if (want_dw && workspace) {
        if (workspace_bytes < need || (uintptr_t)workspace % 16)
            return layer_fail(LA_ERR_INVALID_ARG, who, "workspace too small or not 16-byte aligned");
        p.partial = static_cast<float *>(workspace);
    } else if (want_dw) {
        e = tc_workspace_alloc(&ws, need, stream);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return layer_fail(LA_ERR_NO_MEMORY, who, "workspace allocation");
        }
        p.partial = static_cast<float *>(ws);
    }
    if (v == 8)
        e = launch_rows<T, sizeof(T) == 2 ? 8 : 4, 1, kBack>(p, (unsigned)blocks, stream);
    else if (v == 4)
        e = launch_rows<T, 4, 1, kBack>(p, (unsigned)blocks, stream);
    else if (v == 2)
        e = launch_rows<T, 2, 2, kBack>(p, (unsigned)blocks, stream);
    else
        e = launch_rows<T, 1, 2, kBack>(p, (unsigned)blocks, stream);
    if (e == cudaSuccess) note_launches(1);
    if (e == cudaSuccess && want_dw) {
        e = tchost::launch_dependent(qk_weight_kernel, 2 * ((p.d + 31) / 32), 1024, 0, stream,
                                     static_cast<const float *>(p.partial), p.blocks_q,
                                     (int)blocks, p.d, p.side[0].dw, p.side[1].dw);
        if (e == cudaSuccess) note_launches(1);
    }
    if (ws) {
        const cudaError_t ef = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e == cudaSuccess ? LA_OK : layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
}

// Checks shared by both directions; fills everything but the tensors.
la_status qk_common(const char *who, Params &p, const void *q_weight, const void *k_weight,
                    int norm, float eps, const la_rope *rope, int B, int Hq, int Hk, int N, int d,
                    la_dtype dtype, la_dtype weight_dtype) {
    if (B < 0 || N < 0 || Hq < 0 || Hk < 0)
        return layer_fail(LA_ERR_INVALID_ARG, who, "negative B, Hq, Hk or N");
    if (d < 1 || d > LA_MAX_D) return layer_fail(LA_ERR_INVALID_ARG, who, "d must be in 1..256");
    if (dtype != LA_F32 && dtype != LA_BF16)
        return layer_fail(LA_ERR_INVALID_ARG, who, "unknown dtype");
    if (norm != 0 && norm != 1) return layer_fail(LA_ERR_INVALID_ARG, who, "norm must be 0 or 1");
    if (norm && !(eps > 0.f && std::isfinite(eps)))
        return layer_fail(LA_ERR_INVALID_ARG, who, "eps must be positive and finite");
    if (!norm && (q_weight || k_weight))
        return layer_fail(LA_ERR_INVALID_ARG, who, "weights need norm");
    if ((q_weight || k_weight) && weight_dtype != LA_F32 && weight_dtype != LA_BF16)
        return layer_fail(LA_ERR_INVALID_ARG, who, "unknown weight dtype");
    if ((double)B * N * ((double)Hq + Hk) > 1e11)
        return layer_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
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
        return layer_fail(LA_ERR_INVALID_ARG, who, "rotary_dim must be even and in 0..d");
    if (rope->interleaved != 0 && rope->interleaved != 1)
        return layer_fail(LA_ERR_INVALID_ARG, who, "interleaved must be 0 or 1");
    if (R == 0) return LA_OK;
    if (!rope->frequencies) return layer_fail(LA_ERR_INVALID_ARG, who, "null frequencies");
    if (rope->positions) {
        if (rope->position_bytes != 4 && rope->position_bytes != 8)
            return layer_fail(LA_ERR_INVALID_ARG, who, "position_bytes must be 4 or 8");
        if (rope->position_stride_b < 0 || rope->position_stride_n < 0)
            return layer_fail(LA_ERR_INVALID_ARG, who, "negative position stride");
        if ((uintptr_t)rope->positions % (uintptr_t)rope->position_bytes)
            return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned positions");
    }
    for (int i = 0; i < R / 2; ++i) {
        const double f = rope->frequencies[i];
        if (!(std::fabs(f) <= 1e9))  // also rejects NaN
            return layer_fail(LA_ERR_INVALID_ARG, who, "frequencies must lie in [-1e9, 1e9]");
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

// Whether every pointer of a side is a multiple of its element's size.
bool elements_aligned(const Side &s, la_dtype dtype, la_dtype weight_dtype) {
    const uintptr_t elem = dtype == LA_F32 ? 4 : 2, w = weight_dtype == LA_BF16 ? 2 : 4;
    return (uintptr_t)s.x % elem == 0 && (uintptr_t)s.dy % elem == 0 &&
           (uintptr_t)s.y % elem == 0 && (uintptr_t)s.w % w == 0 && (uintptr_t)s.dw % 4 == 0;
}

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
        if (!s.x || !s.y) return layer_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
        if (!elements_aligned(s, dtype, weight_dtype))
            return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
        if (negative(s.sx) || negative(s.sy))
            return layer_fail(LA_ERR_INVALID_ARG, who, "negative stride");
        if (!rows_disjoint(s.sy, B, s.H, N, d))
            return layer_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
        if (s.y == s.x && !same(s.sx, s.sy))
            return layer_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
    }
    if (B == 0 || N == 0 || Hq + Hk == 0) return LA_OK;
    if (Hq && Hk && (q_out == k || k_out == q || q_out == k_out))
        return layer_fail(LA_ERR_INVALID_ARG, who, "an output aliases the other side");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == LA_F32 ? launch<float, false>(who, p, nullptr, 0, s)
                           : launch<__nv_bfloat16, false>(who, p, nullptr, 0, s);
}

__attribute__((visibility("default")))
la_status la_backward_qk_norm_rope(const void *dq_out, const void *dk_out, const void *q,
                                   const void *k, void *dq, void *dk, float *dq_weight,
                                   float *dk_weight, const la_strides *strides,
                                   const void *q_weight, const void *k_weight, int norm,
                                   float eps, const la_rope *rope, int B, int Hq, int Hk, int N,
                                   int d, la_dtype dtype, la_dtype weight_dtype, void *workspace,
                                   size_t workspace_bytes, la_stream_t stream) {
    const char *who = "la_backward_qk_norm_rope";
    Params p;
    la_status st = qk_common(who, p, q_weight, k_weight, norm, eps, rope, B, Hq, Hk, N, d, dtype,
                             weight_dtype);
    if (st != LA_OK) return st;
    if (!norm && (dq_weight || dk_weight))
        return layer_fail(LA_ERR_INVALID_ARG, who, "weight gradients need norm");
    if (dq_weight && dq_weight == dk_weight)
        return layer_fail(LA_ERR_INVALID_ARG, who, "one buffer for both weight gradients");
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
            return layer_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
        if (!elements_aligned(sd, dtype, weight_dtype))
            return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
        if (negative(sd.sx) || negative(sd.sy) || negative(sd.sdy))
            return layer_fail(LA_ERR_INVALID_ARG, who, "negative stride");
        if (!rows_disjoint(sd.sy, B, sd.H, N, d))
            return layer_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
        if (sd.y == sd.dy && !same(sd.sdy, sd.sy))
            return layer_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
        if (norm && (sd.y == xin[0] || sd.y == xin[1]))
            return layer_fail(LA_ERR_INVALID_ARG, who, "an output aliases an input");
    }
    if (B && N && Hq && Hk && (dq == dk_out || dk == dq_out || dq == dk))
        return layer_fail(LA_ERR_INVALID_ARG, who, "an output aliases the other side");
    // a side without rows has a zero weight gradient
    for (int i = 0; i < 2; ++i)
        if (dw[i] && !p.side[i].dw) {
            const cudaError_t e = cudaMemsetAsync(dw[i], 0, sizeof(float) * d, s);
            if (e != cudaSuccess) return layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
        }
    if (B == 0 || N == 0 || Hq + Hk == 0) return LA_OK;
    if (!norm) {  // turned back and nothing else: the forward of the other sense
        for (Side &sd : p.side) {
            sd.x = sd.dy;
            sd.sx = sd.sdy;
            sd.dy = nullptr;
        }
        for (int i = 0; i < p.half; ++i) p.turns[i] = 0 - p.turns[i];
        return dtype == LA_F32 ? launch<float, false>(who, p, nullptr, 0, s)
                               : launch<__nv_bfloat16, false>(who, p, nullptr, 0, s);
    }
    return dtype == LA_F32 ? launch<float, true>(who, p, workspace, workspace_bytes, s)
                           : launch<__nv_bfloat16, true>(who, p, workspace, workspace_bytes, s);
}

__attribute__((visibility("default")))
size_t la_backward_qk_norm_rope_workspace_bytes(int d) {
    if (d < 1 || d > LA_MAX_D) return 0;
    int sms = 0;
    if (tchost::sm_count(&sms) != cudaSuccess || sms <= 0) sms = 1;
    return sizeof(float) * (size_t)resident_blocks(sms) * d;
}

}  // extern "C"

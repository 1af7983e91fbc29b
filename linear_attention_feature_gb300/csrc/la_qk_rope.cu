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

#include <cmath>
#include <cstdio>

#include "la_internal.h"
#include "la_tc.h"
#include "la_tc_host.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
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
    float eps;
    float *partial;  // backward: [2][gridDim.x][d] sums of g n, or NULL
    unsigned long long turns[kMaxPairs];  // frequency, 2^-64 turns per position
};

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float *p, float x) { *p = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// One warp per row; lane l takes the pairs l, l + 32, ...  Pairs from `half`
// on are neighbours that pass without rotation (the last may be a single).
template <typename T, bool kBack>
__global__ void __launch_bounds__(kThreads) qk_rows_kernel(const __grid_constant__ Params p) {
    constexpr int K = kMaxPairs / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int H = p.side[0].H + p.side[1].H;
    const long long rows = (long long)p.B * p.N * H;
    const int pairs = (p.d + 1) / 2;
    float dw[2][K][2] = {};
    for (long long row = (long long)blockIdx.x * kWarps + warp; row < rows;
         row += (long long)gridDim.x * kWarps) {
        const long long tok = row / H;
        int h = (int)(row % H);
        const int b = (int)(tok / p.N), n = (int)(tok % p.N);
        const int which = h >= p.side[0].H;
        const Side &sd = p.side[which];
        if (which) h -= p.side[0].H;
        const T *x = static_cast<const T *>(sd.x) + b * sd.sx.b + h * sd.sx.h + n * sd.sx.n;
        const T *dy = static_cast<const T *>(sd.dy) + b * sd.sdy.b + h * sd.sdy.h + n * sd.sdy.n;
        T *y = static_cast<T *>(sd.y) + b * sd.sy.b + h * sd.sy.h + n * sd.sy.n;
        const long long pos = position_of(p, b, n);
        float v[K][2], g[K][2], w[K][2], cs[K][2];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int i = lane + 32 * j;
            const bool rot = i < p.half;
            const int lo = rot && !p.interleaved ? i : 2 * i;
            const int hi = rot && !p.interleaved ? i + p.half : 2 * i + 1;
            const bool l_ok = i < pairs, h_ok = i < pairs && hi < p.d;
            v[j][0] = l_ok && (!kBack || p.norm) ? ld(x + lo) : 0.f;
            v[j][1] = h_ok && (!kBack || p.norm) ? ld(x + hi) : 0.f;
            w[j][0] = l_ok ? weight_at(sd.w, p.w_bf16, lo) : 0.f;
            w[j][1] = h_ok ? weight_at(sd.w, p.w_bf16, hi) : 0.f;
            cs[j][0] = 1.f;
            cs[j][1] = 0.f;
            if (rot) turn_of(pos, p.turns[i], &cs[j][0], &cs[j][1]);
            ss += v[j][0] * v[j][0] + v[j][1] * v[j][1];
            if (kBack) {
                const float a = l_ok ? ld(dy + lo) : 0.f, c = h_ok ? ld(dy + hi) : 0.f;
                g[j][0] = a * cs[j][0] + c * cs[j][1];
                g[j][1] = c * cs[j][0] - a * cs[j][1];
                dot += v[j][0] * w[j][0] * g[j][0] + v[j][1] * w[j][1] * g[j][1];
            }
        }
        float r = 1.f;
        if (p.norm) r = rsqrtf(warp_sum(ss) / (float)p.d + p.eps);
        float m = 0.f;
        if (kBack && p.norm) m = warp_sum(dot) * r * r / (float)p.d;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int i = lane + 32 * j;
            const bool rot = i < p.half;
            const int lo = rot && !p.interleaved ? i : 2 * i;
            const int hi = rot && !p.interleaved ? i + p.half : 2 * i + 1;
            float o0, o1;
            if (!kBack) {
                const float a = v[j][0] * r * w[j][0], c = v[j][1] * r * w[j][1];
                o0 = a * cs[j][0] - c * cs[j][1];
                o1 = c * cs[j][0] + a * cs[j][1];
            } else {
                dw[which][j][0] += g[j][0] * v[j][0] * r;
                dw[which][j][1] += g[j][1] * v[j][1] * r;
                o0 = r * (w[j][0] * g[j][0] - v[j][0] * m);
                o1 = r * (w[j][1] * g[j][1] - v[j][1] * m);
            }
            if (i < pairs) {
                st(y + lo, o0);
                if (hi < p.d) st(y + hi, o1);
            }
        }
    }
    if (!kBack || !p.partial) return;
    __shared__ float sum[kWarps][LA_MAX_D];
    for (int s = 0; s < 2; ++s) {
        if (!p.side[s].dw) continue;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int i = lane + 32 * j;
            const bool rot = i < p.half && !p.interleaved;
            const int lo = rot ? i : 2 * i, hi = rot ? i + p.half : 2 * i + 1;
            if (i < pairs) sum[warp][lo] = dw[s][j][0];
            if (i < pairs && hi < p.d) sum[warp][hi] = dw[s][j][1];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.d; i += kThreads) {
            float t = 0.f;
            for (int q = 0; q < kWarps; ++q) t += sum[q][i];
            p.partial[((long long)s * gridDim.x + blockIdx.x) * p.d + i] = t;
        }
    }
}

// dw[i] = the sum of the blocks' partial sums, in block order.
__global__ void qk_weight_kernel(const float *partial, int blocks, int d, float *dwq, float *dwk) {
    float *dw = blockIdx.x ? dwk : dwq;
    const int i = threadIdx.x;
    if (!dw || i >= d) return;
    float t = 0.f;
    for (int b = 0; b < blocks; ++b) t += partial[((long long)blockIdx.x * blocks + b) * d + i];
    dw[i] = t;
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

template <typename T, bool kBack>
la_status launch(const char *who, Params &p, cudaStream_t stream) {
    const long long rows = (long long)p.B * p.N * (p.side[0].H + p.side[1].H);
    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e != cudaSuccess) return qk_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    const int blocks = (int)std::min<long long>((rows + kWarps - 1) / kWarps, 4LL * sms);
    void *ws = nullptr;
    const bool want_dw = kBack && (p.side[0].dw || p.side[1].dw);
    if (want_dw) {
        e = tc_workspace_alloc(&ws, sizeof(float) * 2 * (size_t)blocks * p.d, stream);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return qk_fail(LA_ERR_NO_MEMORY, who, "workspace allocation");
        }
        p.partial = static_cast<float *>(ws);
    }
    qk_rows_kernel<T, kBack><<<blocks, kThreads, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e == cudaSuccess) note_launches(1);
    if (e == cudaSuccess && want_dw) {
        qk_weight_kernel<<<2, LA_MAX_D, 0, stream>>>(p.partial, blocks, p.d, p.side[0].dw,
                                                     p.side[1].dw);
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
    if ((double)B * N * ((double)Hq + Hk) > 1e18)
        return qk_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
    p = Params{};
    p.B = B;
    p.N = N;
    p.d = d;
    p.norm = norm;
    p.eps = eps;
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

// The gated linear recurrence with a gate per channel, forward, backward and
// one token at a time (la_forward_recurrence, la_backward_recurrence,
// la_decode_step_recurrence in include/linattn.h):
//   h_t = a_t h_{t-1} + c_t x_t,   c_t = 1, or 1 - a_t with complement;
// backwards, with e_t = a_{t+1} g_{t+1} what reaches token t from later ones,
//   g_t = dout_t + e_t,  e_{t-1} = a_t g_t,
//   dx_t = c_t g_t,  dgate_t = s_t g_t (h_{t-1} - [complement] x_t),
// s_t = da_t / dgate_t.  Both directions are one affine scan per channel:
// state <- a (state + y) or a state + y.
#include <cuda_bf16.h>

#include <cstdio>

#include "la_internal.h"
#include "la_tc_host.h"

namespace la {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float *p, float x) { *p = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// The gate a and 1 - a (without cancellation where the gate's form allows).
__device__ __forceinline__ void gate_of(int kind, float z, float *a, float *rest) {
    if (kind == LA_GATE_VALUE) {
        *a = z;
        *rest = 1.f - z;
    } else if (kind == LA_GATE_LOG) {
        *a = expf(z);
        *rest = -expm1f(z);
    } else {
        *a = 1.f / (1.f + expf(-z));
        *rest = 1.f / (1.f + expf(z));
    }
}

struct Seq {
    const void *p;
    long long b, n;
};
struct SeqOut {
    void *p;
    long long b, n;
};

struct FwdParams {
    Seq x, gates;
    SeqOut out;
    const float *h0;
    float *h_last;
    int B, N, C, gate, complement;
};

struct BwdParams {
    Seq dout, gates, out, x;
    SeqOut dx, dgates;
    const float *h0, *dh_last;
    float *dh0;
    int B, N, C, gate, complement;
};

// One thread per sequence and channel.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads) rec_forward_kernel(const FwdParams p) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)p.B * p.C) return;
    const int b = (int)(i / p.C), c = (int)(i % p.C);
    const T *x = static_cast<const T *>(p.x.p) + b * p.x.b + c;
    const G *z = static_cast<const G *>(p.gates.p) + b * p.gates.b + c;
    T *out = static_cast<T *>(p.out.p) + b * p.out.b + c;
    float h = p.h0 ? p.h0[i] : 0.f;
    for (int t = 0; t < p.N; ++t) {
        float a, rest;
        gate_of(p.gate, ld(z + t * p.gates.n), &a, &rest);
        const float v = ld(x + t * p.x.n);
        h = fmaf(a, h, p.complement ? rest * v : v);
        st(out + t * p.out.n, h);
    }
    if (p.h_last) p.h_last[i] = h;
}

template <typename T, typename G>
__global__ void __launch_bounds__(kThreads) rec_backward_kernel(const BwdParams p) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)p.B * p.C) return;
    const int b = (int)(i / p.C), c = (int)(i % p.C);
    const T *dout = static_cast<const T *>(p.dout.p) + b * p.dout.b + c;
    const G *z = static_cast<const G *>(p.gates.p) + b * p.gates.b + c;
    const T *out = static_cast<const T *>(p.out.p) + b * p.out.b + c;
    const T *x = static_cast<const T *>(p.x.p) + b * p.x.b + c;
    T *dx = static_cast<T *>(p.dx.p) + b * p.dx.b + c;
    G *dz = static_cast<G *>(p.dgates.p) + b * p.dgates.b + c;
    const float h0 = p.h0 ? p.h0[i] : 0.f;
    float e = p.dh_last ? p.dh_last[i] : 0.f;
    for (int t = p.N - 1; t >= 0; --t) {
        float a, rest;
        gate_of(p.gate, ld(z + t * p.gates.n), &a, &rest);
        const float g = ld(dout + t * p.dout.n) + e;
        float h = t ? ld(out + (t - 1) * p.out.n) : h0;
        if (p.complement) h -= ld(x + t * p.x.n);
        const float slope = p.gate == LA_GATE_VALUE ? 1.f : p.gate == LA_GATE_LOG ? a : a * rest;
        st(dx + t * p.dx.n, p.complement ? rest * g : g);
        st(dz + t * p.dgates.n, slope * g * h);
        e = a * g;
    }
    if (p.dh0) p.dh0[i] = e;
}

template <typename T, typename G>
__global__ void __launch_bounds__(kThreads)
rec_step_kernel(const float *h, float *h_out, const FwdParams p) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)p.B * p.C) return;
    const int b = (int)(i / p.C), c = (int)(i % p.C);
    float a, rest;
    gate_of(p.gate, ld(static_cast<const G *>(p.gates.p) + b * p.gates.b + c), &a, &rest);
    const float v = ld(static_cast<const T *>(p.x.p) + b * p.x.b + c);
    const float s = fmaf(a, h[i], p.complement ? rest * v : v);
    h_out[i] = s;
    st(static_cast<T *>(p.out.p) + b * p.out.b + c, s);
}

la_status rec_fail(la_status s, const char *who, const char *msg) {
    char text[200];
    std::snprintf(text, sizeof(text), "%s: %s", who, msg);
    set_last_error(text);
    return s;
}

la_status rec_common(const char *who, int B, int N, int C, la_gate gate, int complement,
                     la_dtype dtype, la_dtype gate_dtype) {
    if (B < 0 || N < 0 || C < 0) return rec_fail(LA_ERR_INVALID_ARG, who, "negative B, N or C");
    if (gate != LA_GATE_VALUE && gate != LA_GATE_LOG && gate != LA_GATE_LOGIT)
        return rec_fail(LA_ERR_INVALID_ARG, who, "unknown gate form");
    if (complement != 0 && complement != 1)
        return rec_fail(LA_ERR_INVALID_ARG, who, "complement must be 0 or 1");
    if (dtype != LA_F32 && dtype != LA_BF16)
        return rec_fail(LA_ERR_INVALID_ARG, who, "unknown dtype");
    if (gate_dtype != LA_F32 && gate_dtype != dtype)
        return rec_fail(LA_ERR_INVALID_ARG, who, "gate_dtype must be LA_F32 or dtype");
    if ((double)B * C > 2147483647.0 * 32)
        return rec_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
    return LA_OK;
}

// Whether no two rows of C elements overlap.
bool rows_disjoint(long long b, long long n, int B, int N, int C) {
    if (B <= 1) return N <= 1 || n >= C;
    if (N <= 1) return b >= C;
    return b >= n ? n >= C && b >= n * (N - 1) + C : b >= C && n >= b * (B - 1) + C;
}

la_seq_strides pick(const la_seq_strides *s, int i, int N, int C) {
    return s ? s[i] : la_seq_strides{(long long)N * C, C};
}

la_status rec_copy(const char *who, float *dst, const float *src, size_t n, cudaStream_t s) {
    if (!dst || dst == src) return LA_OK;
    const cudaError_t e =
        src ? cudaMemcpyAsync(dst, src, sizeof(float) * n, cudaMemcpyDeviceToDevice, s)
            : cudaMemsetAsync(dst, 0, sizeof(float) * n, s);
    return e == cudaSuccess ? LA_OK : rec_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
}

unsigned blocks_for(int B, int C) {
    return (unsigned)(((long long)B * C + kThreads - 1) / kThreads);
}

la_status done(const char *who) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return rec_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    note_launches(1);
    return LA_OK;
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

__attribute__((visibility("default")))
la_status la_forward_recurrence(const void *x, const void *gates, const float *h0, void *out,
                                float *h_last, const la_seq_strides *strides, int B, int N, int C,
                                la_gate gate, int complement, la_dtype dtype, la_dtype gate_dtype,
                                la_stream_t stream) {
    const char *who = "la_forward_recurrence";
    la_status st = rec_common(who, B, N, C, gate, complement, dtype, gate_dtype);
    if (st != LA_OK) return st;
    if (B == 0 || C == 0) return LA_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) return rec_copy(who, h_last, h0, (size_t)B * C, s);
    if (!x || !gates || !out) return rec_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
    const la_seq_strides sx = pick(strides, 0, N, C), sg = pick(strides, 1, N, C),
                         so = pick(strides, 2, N, C);
    if (sx.b < 0 || sx.n < 0 || sg.b < 0 || sg.n < 0 || so.b < 0 || so.n < 0)
        return rec_fail(LA_ERR_INVALID_ARG, who, "negative stride");
    if (!rows_disjoint(so.b, so.n, B, N, C))
        return rec_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
    if (out == gates) return rec_fail(LA_ERR_INVALID_ARG, who, "out aliases gates");
    if (out == x && (sx.b != so.b || sx.n != so.n))
        return rec_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
    const FwdParams p{{x, sx.b, sx.n}, {gates, sg.b, sg.n}, {out, so.b, so.n}, h0, h_last, B, N, C,
                      gate, complement};
    const unsigned nb = blocks_for(B, C);
    if (dtype == LA_F32)
        rec_forward_kernel<float, float><<<nb, kThreads, 0, s>>>(p);
    else if (gate_dtype == LA_F32)
        rec_forward_kernel<__nv_bfloat16, float><<<nb, kThreads, 0, s>>>(p);
    else
        rec_forward_kernel<__nv_bfloat16, __nv_bfloat16><<<nb, kThreads, 0, s>>>(p);
    return done(who);
}

__attribute__((visibility("default")))
la_status la_backward_recurrence(const void *dout, const void *gates, const void *out,
                                 const void *x, const float *h0, const float *dh_last, void *dx,
                                 void *dgates, float *dh0, const la_seq_strides *strides, int B,
                                 int N, int C, la_gate gate, int complement, la_dtype dtype,
                                 la_dtype gate_dtype, la_stream_t stream) {
    const char *who = "la_backward_recurrence";
    la_status st = rec_common(who, B, N, C, gate, complement, dtype, gate_dtype);
    if (st != LA_OK) return st;
    if (B == 0 || C == 0) return LA_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) return rec_copy(who, dh0, dh_last, (size_t)B * C, s);
    if (!dout || !gates || !out || !dx || !dgates || (complement && !x))
        return rec_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
    la_seq_strides ss[6];
    for (int i = 0; i < 6; ++i) {
        if (i == 3 && !complement) {
            ss[i] = {0, 0};
            continue;
        }
        ss[i] = pick(strides, i, N, C);
        if (ss[i].b < 0 || ss[i].n < 0)
            return rec_fail(LA_ERR_INVALID_ARG, who, "negative stride");
        if (i >= 4 && !rows_disjoint(ss[i].b, ss[i].n, B, N, C))
            return rec_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
    }
    if (dx == gates || dx == out || (complement && dx == x) || dx == dgates || dgates == dout ||
        dgates == gates || dgates == out || (complement && dgates == x))
        return rec_fail(LA_ERR_INVALID_ARG, who, "an output aliases another tensor");
    if (dx == dout && (ss[0].b != ss[4].b || ss[0].n != ss[4].n))
        return rec_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
    const BwdParams p{{dout, ss[0].b, ss[0].n},
                      {gates, ss[1].b, ss[1].n},
                      {out, ss[2].b, ss[2].n},
                      {complement ? x : nullptr, ss[3].b, ss[3].n},
                      {dx, ss[4].b, ss[4].n},
                      {dgates, ss[5].b, ss[5].n},
                      h0,
                      dh_last,
                      dh0,
                      B,
                      N,
                      C,
                      gate,
                      complement};
    const unsigned nb = blocks_for(B, C);
    if (dtype == LA_F32)
        rec_backward_kernel<float, float><<<nb, kThreads, 0, s>>>(p);
    else if (gate_dtype == LA_F32)
        rec_backward_kernel<__nv_bfloat16, float><<<nb, kThreads, 0, s>>>(p);
    else
        rec_backward_kernel<__nv_bfloat16, __nv_bfloat16><<<nb, kThreads, 0, s>>>(p);
    return done(who);
}

__attribute__((visibility("default")))
la_status la_decode_step_recurrence(const float *h, float *h_out, const void *x, const void *gates,
                                    void *out, const long long *strides, int B, int C,
                                    la_gate gate, int complement, la_dtype dtype,
                                    la_dtype gate_dtype, la_stream_t stream) {
    const char *who = "la_decode_step_recurrence";
    la_status st = rec_common(who, B, 1, C, gate, complement, dtype, gate_dtype);
    if (st != LA_OK) return st;
    if (B == 0 || C == 0) return LA_OK;
    if (!h || !h_out || !x || !gates || !out)
        return rec_fail(LA_ERR_INVALID_ARG, who, "null pointer");
    const long long sx = strides ? strides[0] : C, sg = strides ? strides[1] : C,
                    so = strides ? strides[2] : C;
    if (sx < 0 || sg < 0 || so < 0) return rec_fail(LA_ERR_INVALID_ARG, who, "negative stride");
    if (!rows_disjoint(so, 0, B, 1, C))
        return rec_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
    if (out == gates || out == h || out == h_out)
        return rec_fail(LA_ERR_INVALID_ARG, who, "out aliases another tensor");
    if (out == x && sx != so)
        return rec_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
    const FwdParams p{{x, sx, 0}, {gates, sg, 0}, {out, so, 0}, nullptr, nullptr, B, 1, C,
                      gate, complement};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned nb = blocks_for(B, C);
    if (dtype == LA_F32)
        rec_step_kernel<float, float><<<nb, kThreads, 0, s>>>(h, h_out, p);
    else if (gate_dtype == LA_F32)
        rec_step_kernel<__nv_bfloat16, float><<<nb, kThreads, 0, s>>>(h, h_out, p);
    else
        rec_step_kernel<__nv_bfloat16, __nv_bfloat16><<<nb, kThreads, 0, s>>>(h, h_out, p);
    return done(who);
}

}  // extern "C"

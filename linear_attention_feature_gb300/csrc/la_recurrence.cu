// The gated linear recurrence with a gate per channel: argument checks, the
// forward scan and the step of one token (la_forward_recurrence,
// la_backward_recurrence, la_decode_step_recurrence in include/linattn.h).  The
// scan itself is in la_recurrence.cuh.
#include <initializer_list>

#include "la_recurrence.cuh"

namespace la {
namespace rec {

la_status launch_backward(const char *who, Params &p, la_gate gate, la_dtype dtype,
                          la_dtype gate_dtype, Workspace ws, cudaStream_t s);

namespace {

constexpr int kStepThreads = 256;

// One token: V adjacent channels per thread, bound by the launch (256 x 4096
// channels: 2.6 us on the device).
struct StepParams {
    const float *h;
    float *h_out;
    const void *x, *gates;
    void *out;
    long long sx, sg, so;
    int B, C, complement;
};

template <typename T, typename G, int V, int kGate>
__global__ void __launch_bounds__(kStepThreads) rec_step_kernel(const StepParams p) {
    const long long i = ((long long)blockIdx.x * kStepThreads + threadIdx.x) * V;
    if (i >= (long long)p.B * p.C) return;
    const int b = (int)(i / p.C), c = (int)(i % p.C);
    auto get = [](const auto *q) {
        using E = std::remove_const_t<std::remove_reference_t<decltype(*q)>>;
        return widen(reinterpret_cast<const Mem<E, V> *>(q));
    };
    const Vec<V> x = get(static_cast<const T *>(p.x) + b * p.sx + c);
    const Vec<V> z = get(static_cast<const G *>(p.gates) + b * p.sg + c);
    const Vec<V> h = get(p.h + i);
    Vec<V> a, rest, s;
    gate_of<kGate, V>(z, p.complement, a, rest);
#pragma unroll
    for (int e = 0; e < V; ++e)
        s.v[e] = fmaf(a.v[e], h.v[e], p.complement ? __fmul_rn(rest.v[e], x.v[e]) : x.v[e]);
    narrow(reinterpret_cast<Mem<float, V> *>(p.h_out + i), s);
    narrow(reinterpret_cast<Mem<T, V> *>(static_cast<T *>(p.out) + b * p.so + c), s);
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

// Whether every pointer (may be NULL) is a multiple of its element's size.
bool elements_aligned(int elem, std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if ((uintptr_t)q % (uintptr_t)elem) return false;
    return true;
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

la_status done(const char *who, cudaError_t e) {
    if (e != cudaSuccess) return rec_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    note_launches(1);
    return LA_OK;
}

template <typename T, typename G, int V>
cudaError_t launch_step(const StepParams &p, la_gate gate, cudaStream_t s) {
    const unsigned nb = (unsigned)(((long long)p.B * p.C / V + kStepThreads - 1) / kStepThreads);
    if (gate == LA_GATE_VALUE)
        rec_step_kernel<T, G, V, LA_GATE_VALUE><<<nb, kStepThreads, 0, s>>>(p);
    else if (gate == LA_GATE_LOG)
        rec_step_kernel<T, G, V, LA_GATE_LOG><<<nb, kStepThreads, 0, s>>>(p);
    else
        rec_step_kernel<T, G, V, LA_GATE_LOGIT><<<nb, kStepThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, typename G>
la_status step(const char *who, const StepParams &p, la_gate gate, cudaStream_t s) {
    // 4 channels per thread where every row allows it
    const bool four = p.C % 4 == 0 && aligned(p.h, 0, 0, 1, 1, 4, 4) &&
                      aligned(p.h_out, 0, 0, 1, 1, 4, 4) &&
                      aligned(p.x, p.sx, 0, p.B, 1, 4, sizeof(T)) &&
                      aligned(p.gates, p.sg, 0, p.B, 1, 4, sizeof(G)) &&
                      aligned(p.out, p.so, 0, p.B, 1, 4, sizeof(T));
    return done(who, four ? launch_step<T, G, 4>(p, gate, s) : launch_step<T, G, 1>(p, gate, s));
}

}  // namespace
}  // namespace rec
}  // namespace la

using namespace la;
using namespace la::rec;

extern "C" {

__attribute__((visibility("default")))
la_status la_forward_recurrence(const void *x, const void *gates, const float *h0, void *out,
                                float *h_last, const la_seq_strides *strides, int B, int N, int C,
                                la_gate gate, int complement, la_dtype dtype, la_dtype gate_dtype,
                                void *workspace, size_t workspace_bytes, la_stream_t stream) {
    const char *who = "la_forward_recurrence";
    la_status st = rec_common(who, B, N, C, gate, complement, dtype, gate_dtype);
    if (st != LA_OK) return st;
    if (B == 0 || C == 0) return LA_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) return rec_copy(who, h_last, h0, (size_t)B * C, s);
    if (!x || !gates || !out) return rec_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
    if (!elements_aligned(dtype == LA_F32 ? 4 : 2, {x, out}) ||
        !elements_aligned(gate_dtype == LA_F32 ? 4 : 2, {gates}) ||
        !elements_aligned(4, {h0, h_last}))
        return rec_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
    const la_seq_strides sx = pick(strides, 0, N, C), sg = pick(strides, 1, N, C),
                         so = pick(strides, 2, N, C);
    if (sx.b < 0 || sx.n < 0 || sg.b < 0 || sg.n < 0 || so.b < 0 || so.n < 0)
        return rec_fail(LA_ERR_INVALID_ARG, who, "negative stride");
    if (!rows_disjoint(so.b, so.n, B, N, C))
        return rec_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
    if (out == gates) return rec_fail(LA_ERR_INVALID_ARG, who, "out aliases gates");
    if (h_last && (h_last == x || h_last == gates || (h_last == out && N > 1)))
        return rec_fail(LA_ERR_INVALID_ARG, who, "h_last aliases a tensor of the sequence");
    if (out == x && (sx.b != so.b || sx.n != so.n))
        return rec_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
    Params p{};
    p.in[0] = {x, sx.b, sx.n};
    p.in[1] = {gates, sg.b, sg.n};
    p.out[0] = {out, so.b, so.n};
    p.first = h0;
    p.last = h_last;
    p.B = B;
    p.N = N;
    p.C = C;
    p.complement = complement;
    return launch<false>(who, p, gate, dtype, gate_dtype, {workspace, workspace_bytes}, s);
}

__attribute__((visibility("default")))
la_status la_backward_recurrence(const void *dout, const void *gates, const void *out,
                                 const void *x, const float *h0, const float *dh_last, void *dx,
                                 void *dgates, float *dh0, const la_seq_strides *strides, int B,
                                 int N, int C, la_gate gate, int complement, la_dtype dtype,
                                 la_dtype gate_dtype, void *workspace, size_t workspace_bytes,
                                 la_stream_t stream) {
    const char *who = "la_backward_recurrence";
    la_status st = rec_common(who, B, N, C, gate, complement, dtype, gate_dtype);
    if (st != LA_OK) return st;
    if (B == 0 || C == 0) return LA_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) return rec_copy(who, dh0, dh_last, (size_t)B * C, s);
    if (!dout || !gates || !out || !dx || !dgates || (complement && !x))
        return rec_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
    if (!elements_aligned(dtype == LA_F32 ? 4 : 2, {dout, out, x, dx}) ||
        !elements_aligned(gate_dtype == LA_F32 ? 4 : 2, {gates, dgates}) ||
        !elements_aligned(4, {h0, dh_last, dh0}))
        return rec_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
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
    if (dh0 && (dh0 == dout || dh0 == gates || dh0 == out || (complement && dh0 == x) ||
                dh0 == dx || dh0 == dgates))
        return rec_fail(LA_ERR_INVALID_ARG, who, "dh0 aliases a tensor of the sequence");
    if (dx == dout && (ss[0].b != ss[4].b || ss[0].n != ss[4].n))
        return rec_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
    Params p{};
    const void *in[4] = {dout, gates, out, complement ? x : nullptr};
    for (int i = 0; i < 4; ++i) p.in[i] = {in[i], ss[i].b, ss[i].n};
    p.out[0] = {dx, ss[4].b, ss[4].n};
    p.out[1] = {dgates, ss[5].b, ss[5].n};
    p.first = dh_last;
    p.last = dh0;
    p.h0 = h0;
    p.B = B;
    p.N = N;
    p.C = C;
    p.complement = complement;
    return launch_backward(who, p, gate, dtype, gate_dtype, {workspace, workspace_bytes}, s);
}

__attribute__((visibility("default")))
size_t la_recurrence_workspace_bytes(int B, int C, la_dtype dtype) {
    if (B < 1 || C < 1 || (dtype != LA_F32 && dtype != LA_BF16)) return 0;
    const long long strips = (C + (dtype == LA_F32 ? 31LL : 63LL)) / (dtype == LA_F32 ? 32 : 64);
    if (B * strips > kFewStrips) return 0;
    return (sizeof(float2) * (kMaxPieces - 1) + sizeof(float)) * (size_t)B * C;
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
    if (!elements_aligned(dtype == LA_F32 ? 4 : 2, {x, out}) ||
        !elements_aligned(gate_dtype == LA_F32 ? 4 : 2, {gates}) ||
        !elements_aligned(4, {h, h_out}))
        return rec_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
    const long long sx = strides ? strides[0] : C, sg = strides ? strides[1] : C,
                    so = strides ? strides[2] : C;
    if (sx < 0 || sg < 0 || so < 0) return rec_fail(LA_ERR_INVALID_ARG, who, "negative stride");
    if (!rows_disjoint(so, 0, B, 1, C))
        return rec_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
    if (out == gates || out == h || out == h_out)
        return rec_fail(LA_ERR_INVALID_ARG, who, "out aliases another tensor");
    if (out == x && sx != so)
        return rec_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
    // over x or the gates each value of the state lies where its own input does, or not
    if ((h_out == x && !(dtype == LA_F32 && (sx == C || B == 1))) ||
        (h_out == gates && !(gate_dtype == LA_F32 && (sg == C || B == 1))))
        return rec_fail(LA_ERR_INVALID_ARG, who, "h_out aliases an input");
    const StepParams p{h, h_out, x, gates, out, sx, sg, so, B, C, complement};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LA_F32) return step<float, float>(who, p, gate, s);
    if (gate_dtype == LA_F32) return step<__nv_bfloat16, float>(who, p, gate, s);
    return step<__nv_bfloat16, __nv_bfloat16>(who, p, gate, s);
}

}  // extern "C"

// The gated linear recurrence with a gate per channel, forward, backward and
// one token at a time (la_forward_recurrence, la_backward_recurrence,
// la_decode_step_recurrence in include/linattn.h):
//   h_t = a_t h_{t-1} + c_t x_t,   c_t = 1, or 1 - a_t with complement;
// backwards, with e_t = a_{t+1} g_{t+1} what reaches token t from later ones,
//   g_t = dout_t + e_t,  e_{t-1} = a_t g_t,
//   dx_t = c_t g_t,  dgate_t = s_t g_t (h_{t-1} - [complement] x_t),
// s_t = da_t / dgate_t.  Both directions are one affine scan per channel,
//   state <- a state + y   (forward),   state <- a (state + y)   (backward),
// walked in scan order: tokens ascending, or descending for the gradient.
//
// The data is read once.  A block of 8 warps takes a strip of 32 lanes x V
// channels (one 128-byte row per token and warp) and walks the sequence in
// rounds of 8 x L tokens, L consecutive ones per warp: each thread copies its own
// tokens of its own channels into shared memory with cp.async, three rounds deep
// (the slots are private to the thread, so the copies need no barrier), forms
// the affine map (A, H) of its L tokens, and one block barrier later applies
// the maps of the warps before it to the state that the block carries from
// round to round, then walks its L tokens again from there and stores.
//
// Where there are fewer strips than the GPU holds blocks, a cluster of S blocks
// shares a strip: a round is then S x 8 x L tokens, each block leaves its map in
// the shared memory of the others, and one cluster barrier replaces the
// sequence's serial chain.  Maps are joined in scan order, the same for every
// alignment and type, so repeated calls are bit-identical.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdio>

#include "la_internal.h"
#include "la_tc_host.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 3;        // rounds of copies in flight
constexpr int kMaxCluster = 8;

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float *p, float x) { *p = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// The gate a and 1 - a, without cancellation in either.
template <int kGate>
__device__ __forceinline__ void gate_of(float z, float *a, float *rest) {
    if (kGate == LA_GATE_VALUE) {
        *a = z;
        *rest = __fsub_rn(1.f, z);
    } else if (kGate == LA_GATE_LOG) {
        *a = expf(z);
        *rest = -expm1f(z);
    } else {
        const float t = expf(-fabsf(z)), s = __fdividef(1.f, 1.f + t), u = __fmul_rn(t, s);
        *a = z < 0.f ? u : s;
        *rest = z < 0.f ? s : u;
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

// Forward: in = {x, gates}, out = {out}.  Backward: in = {dout, gates, out, x},
// out = {dx, dgates}.
struct Params {
    Seq in[4];
    SeqOut out[2];
    const float *first;  // h0; backward dh_last: the carried state at the start
    float *last;         // h_last; backward dh0
    const float *h0;     // backward: h_0, for the first token's gate
    int B, N, C, complement, strips;
};

__device__ __forceinline__ void copy_async(void *dst, const void *src, int bytes, int valid) {
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    if (bytes == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(valid)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(valid)
                     : "memory");
}

// V adjacent values in a thread's slot.
template <typename T, int V>
struct alignas(sizeof(T) * V) Slot {
    T v[V];
};

// Slots of one tensor in one stage: [L][kThreads].
template <typename T, int V, int L>
constexpr int slots_bytes() {
    return (int)sizeof(T) * V * L * kThreads;
}
template <typename T, typename G, int V, int L, bool kBack>
constexpr int stage_bytes(int complement) {
    return slots_bytes<T, V, L>() * (kBack ? 2 + complement : 1) + slots_bytes<G, V, L>();
}

// kFast: every row of every tensor is aligned to V values.
template <typename T, typename G, int V, int L, int kGate, bool kFast, bool kBack>
__global__ void __launch_bounds__(kThreads, 2) rec_scan_kernel(const __grid_constant__ Params p) {
    namespace cg = cooperative_groups;
    constexpr int kTile = kWarps * L;  // tokens per block and round
    extern __shared__ char stages[];
    __shared__ float warp_map[2][kWarps][2][32 * V];
    __shared__ float block_map[2][kMaxCluster][2][32 * V];

    const cg::cluster_group cluster = cg::this_cluster();
    const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int strip = (int)(blockIdx.x / S) % p.strips, b = (int)(blockIdx.x / S) / p.strips;
    const int c = (strip * 32 + lane) * V;          // first channel
    const int here = min(max(p.C - c, 0), V);       // channels that exist
    const int rounds = (int)(((long long)p.N + (long long)S * kTile - 1) / ((long long)S * kTile));
    const int bytes = stage_bytes<T, G, V, L, kBack>(p.complement);

    // token of this thread's i-th step in scan order in round r, or outside
    // [0, N) behind the sequence's end
    auto first_step = [&](int r) { return ((long long)r * S + rank) * kTile + warp * L; };
    auto token = [&](long long step) { return kBack ? p.N - 1 - step : step; };

    auto slot_x = [&](int stage, int which) {
        return reinterpret_cast<Slot<T, V> *>(stages + (size_t)stage * bytes +
                                              slots_bytes<G, V, L>() +
                                              which * slots_bytes<T, V, L>()) + tid;
    };
    auto slot_z = [&](int stage) {
        return reinterpret_cast<Slot<G, V> *>(stages + (size_t)stage * bytes) + tid;
    };
    auto fetch_one = [&](auto *slot, const Seq &q, long long t, bool ok) {
        using E = std::remove_reference_t<decltype(slot->v[0])>;
        const E *src = static_cast<const E *>(q.p) + (ok ? b * q.b + t * q.n + c : 0);
        if (kFast) {
            copy_async(slot, src, (int)sizeof(E) * V, ok ? here * (int)sizeof(E) : 0);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) slot->v[e] = ok && e < here ? src[e] : E(0.f);
        }
    };
    auto fetch = [&](int r) {
        const int stage = r % kStages;
        const long long s0 = first_step(r);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const long long t = token(s0 + i);
            const bool ok = r < rounds && s0 + i < p.N && here > 0;
            if (ok || kFast) {
                fetch_one(slot_x(stage, 0) + i * kThreads, p.in[0], t, ok);
                fetch_one(slot_z(stage) + i * kThreads, p.in[1], t, ok);
                if (kBack) {
                    fetch_one(slot_x(stage, 1) + i * kThreads, p.in[2], t - 1, ok && t > 0);
                    if (p.complement) fetch_one(slot_x(stage, 2) + i * kThreads, p.in[3], t, ok);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

#pragma unroll
    for (int r = 0; r < kStages; ++r) fetch(r);

    float carry[V], h0[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long at = (long long)b * p.C + c + e;
        carry[e] = p.first && e < here ? p.first[at] : 0.f;
        h0[e] = kBack && p.h0 && e < here ? p.h0[at] : 0.f;
    }

    // the others' shared memory is written from here on
    if (S > 1) cluster.sync();
    for (int r = 0; r < rounds; ++r) {
        const int stage = r % kStages, par = r & 1;
        const long long s0 = first_step(r);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        // a and y (backward: a and 1 - a) of the L tokens, and their map
        float a[L][V], y[L][V], A[V], H[V];
#pragma unroll
        for (int e = 0; e < V; ++e) A[e] = 1.f, H[e] = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const Slot<T, V> in = slot_x(stage, 0)[i * kThreads];
            const Slot<G, V> z = slot_z(stage)[i * kThreads];
            const bool ok = s0 + i < p.N;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float rest;
                const float v = ld(&in.v[e]);
                gate_of<kGate>(ld(&z.v[e]), &a[i][e], &rest);
                if (!kBack) y[i][e] = p.complement ? __fmul_rn(rest, v) : v;
                if (kBack) y[i][e] = rest;
                if (!ok) a[i][e] = 1.f, y[i][e] = 0.f;
                H[e] = kBack ? __fmul_rn(a[i][e], __fadd_rn(ok ? v : 0.f, H[e]))
                             : fmaf(a[i][e], H[e], y[i][e]);
                A[e] = __fmul_rn(A[e], a[i][e]);
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            warp_map[par][warp][0][lane * V + e] = A[e];
            warp_map[par][warp][1][lane * V + e] = H[e];
        }
        __syncthreads();
        // the map of the warps before this one, and of the whole block
        float Ab[V], Hb[V];
#pragma unroll
        for (int e = 0; e < V; ++e) Ab[e] = 1.f, Hb[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (w == warp) A[e] = Ab[e], H[e] = Hb[e];
                const float Aw = warp_map[par][w][0][lane * V + e];
                Hb[e] = fmaf(Aw, Hb[e], warp_map[par][w][1][lane * V + e]);
                Ab[e] = __fmul_rn(Ab[e], Aw);
            }
        }
        float state[V];
        if (S == 1) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                state[e] = fmaf(A[e], carry[e], H[e]);
                carry[e] = fmaf(Ab[e], carry[e], Hb[e]);
            }
        } else {
            for (int to = warp; to < S; to += kWarps) {
                float *there = cluster.map_shared_rank(&block_map[par][rank][0][0], to);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    there[lane * V + e] = Ab[e];
                    there[32 * V + lane * V + e] = Hb[e];
                }
            }
            cluster.sync();
            for (int k = 0; k < S; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (k == rank) state[e] = fmaf(A[e], carry[e], H[e]);
                    carry[e] = fmaf(block_map[par][k][0][lane * V + e], carry[e],
                                    block_map[par][k][1][lane * V + e]);
                }
        }
        // the L tokens again, from the state that reaches them
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const bool ok = s0 + i < p.N && here > 0;
            const long long t = token(s0 + i);
            float o[V], oz[V];
            if (!kBack) {
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = state[e] = fmaf(a[i][e], state[e], y[i][e]);
            } else {
                const Slot<T, V> in = slot_x(stage, 0)[i * kThreads];
                const Slot<T, V> h = slot_x(stage, 1)[i * kThreads];
                const Slot<T, V> x = slot_x(stage, p.complement ? 2 : 0)[i * kThreads];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float g = __fadd_rn(ok ? ld(&in.v[e]) : 0.f, state[e]);
                    float before = t > 0 ? ld(&h.v[e]) : h0[e];
                    if (p.complement) before = __fsub_rn(before, ld(&x.v[e]));
                    const float slope = kGate == LA_GATE_VALUE ? 1.f
                                        : kGate == LA_GATE_LOG ? a[i][e]
                                                               : __fmul_rn(a[i][e], y[i][e]);
                    o[e] = p.complement ? __fmul_rn(y[i][e], g) : g;
                    oz[e] = __fmul_rn(__fmul_rn(slope, g), before);
                    state[e] = __fmul_rn(a[i][e], g);
                }
            }
            if (!ok) continue;
            auto put = [&](auto *base, const SeqOut &q, const float (&v)[V]) {
                using E = std::remove_pointer_t<decltype(base)>;
                E *dst = base + b * q.b + t * q.n + c;
                if (kFast && here == V) {
                    Slot<E, V> w;
#pragma unroll
                    for (int e = 0; e < V; ++e) st(&w.v[e], v[e]);
                    *reinterpret_cast<Slot<E, V> *>(dst) = w;
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (e < here) st(dst + e, v[e]);
                }
            };
            put(static_cast<T *>(p.out[0].p), p.out[0], o);
            if (kBack) put(static_cast<G *>(p.out[1].p), p.out[1], oz);
        }
        // the state behind the last token, as its warp has it: forward, these
        // are the bits that `out` was rounded from
        if (p.last && s0 < p.N && s0 + L >= p.N)
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < here) p.last[(long long)b * p.C + c + e] = state[e];
        fetch(r + kStages);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// One token: V adjacent channels per thread.
struct StepParams {
    const float *h;
    float *h_out;
    const void *x, *gates;
    void *out;
    long long sx, sg, so;
    int B, C, complement;
};

template <typename T, typename G, int V, int kGate>
__global__ void __launch_bounds__(kThreads) rec_step_kernel(const StepParams p) {
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * V;
    if (i >= (long long)p.B * p.C) return;
    const int b = (int)(i / p.C), c = (int)(i % p.C);
    const Slot<T, V> x = *reinterpret_cast<const Slot<T, V> *>(static_cast<const T *>(p.x) + b * p.sx + c);
    const Slot<G, V> z = *reinterpret_cast<const Slot<G, V> *>(static_cast<const G *>(p.gates) + b * p.sg + c);
    const Slot<float, V> h = *reinterpret_cast<const Slot<float, V> *>(p.h + i);
    Slot<float, V> s;
    Slot<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float a, rest;
        const float v = ld(&x.v[e]);
        gate_of<kGate>(ld(&z.v[e]), &a, &rest);
        s.v[e] = fmaf(a, h.v[e], p.complement ? __fmul_rn(rest, v) : v);
        st(&o.v[e], s.v[e]);
    }
    *reinterpret_cast<Slot<float, V> *>(p.h_out + i) = s;
    *reinterpret_cast<Slot<T, V> *>(static_cast<T *>(p.out) + b * p.so + c) = o;
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

la_status done(const char *who, cudaError_t e) {
    if (e != cudaSuccess) return rec_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    note_launches(1);
    return LA_OK;
}

bool aligned(const void *p, long long b, long long n, int B, int N, int v, int elem) {
    return (uintptr_t)p % (uintptr_t)(v * elem) == 0 && (B <= 1 || b % v == 0) &&
           (N <= 1 || n % v == 0);
}

template <typename T, typename G, int V, int kGate, bool kFast, bool kBack>
cudaError_t launch_scan(Params p, cudaStream_t stream) {
    constexpr int L = kBack ? 8 : 16;
    auto kern = rec_scan_kernel<T, G, V, L, kGate, kFast, kBack>;
    const size_t smem = (size_t)kStages * stage_bytes<T, G, V, L, kBack>(p.complement);
    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    p.strips = (p.C + 32 * V - 1) / (32 * V);
    const long long strips = (long long)p.B * p.strips;
    // as many blocks per strip as the GPU holds at once (two per SM) and the
    // sequence has work for
    int S = 1;
    while (S < kMaxCluster && strips * S * 2 <= 2LL * sms && (long long)S * kWarps * L < p.N) S *= 2;
    if (strips * S > 2147483647LL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(strips * S));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)S, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, typename G, int V, bool kFast, bool kBack>
cudaError_t launch_gate(const Params &p, la_gate gate, cudaStream_t s) {
    if (gate == LA_GATE_VALUE) return launch_scan<T, G, V, LA_GATE_VALUE, kFast, kBack>(p, s);
    if (gate == LA_GATE_LOG) return launch_scan<T, G, V, LA_GATE_LOG, kFast, kBack>(p, s);
    return launch_scan<T, G, V, LA_GATE_LOGIT, kFast, kBack>(p, s);
}

template <bool kBack>
la_status launch(const char *who, const Params &p, la_gate gate, la_dtype dtype,
                 la_dtype gate_dtype, cudaStream_t s) {
    // the kernel takes 4 bytes of x per thread and token: two bf16 channels
    const int v = dtype == LA_F32 ? 1 : 2;
    const int ex = dtype == LA_F32 ? 4 : 2, ez = gate_dtype == LA_F32 ? 4 : 2;
    bool fast = true;
    for (int i = 0; i < 4; ++i)
        fast = fast && aligned(p.in[i].p, p.in[i].b, p.in[i].n, p.B, p.N, v, i == 1 ? ez : ex);
    for (int i = 0; i < 2; ++i)
        fast = fast && aligned(p.out[i].p, p.out[i].b, p.out[i].n, p.B, p.N, v, i == 1 ? ez : ex);
    using bf16 = __nv_bfloat16;
    cudaError_t e;
    if (dtype == LA_F32)
        e = launch_gate<float, float, 1, true, kBack>(p, gate, s);
    else if (gate_dtype == LA_F32)
        e = fast ? launch_gate<bf16, float, 2, true, kBack>(p, gate, s)
                 : launch_gate<bf16, float, 2, false, kBack>(p, gate, s);
    else
        e = fast ? launch_gate<bf16, bf16, 2, true, kBack>(p, gate, s)
                 : launch_gate<bf16, bf16, 2, false, kBack>(p, gate, s);
    return done(who, e);
}

template <typename T, typename G, int V>
cudaError_t launch_step(const StepParams &p, la_gate gate, cudaStream_t s) {
    const unsigned nb = (unsigned)(((long long)p.B * p.C / V + kThreads - 1) / kThreads);
    if (gate == LA_GATE_VALUE)
        rec_step_kernel<T, G, V, LA_GATE_VALUE><<<nb, kThreads, 0, s>>>(p);
    else if (gate == LA_GATE_LOG)
        rec_step_kernel<T, G, V, LA_GATE_LOG><<<nb, kThreads, 0, s>>>(p);
    else
        rec_step_kernel<T, G, V, LA_GATE_LOGIT><<<nb, kThreads, 0, s>>>(p);
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
    return launch<false>(who, p, gate, dtype, gate_dtype, s);
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
    return launch<true>(who, p, gate, dtype, gate_dtype, s);
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
    const StepParams p{h, h_out, x, gates, out, sx, sg, so, B, C, complement};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LA_F32) return step<float, float>(who, p, gate, s);
    if (gate_dtype == LA_F32) return step<__nv_bfloat16, float>(who, p, gate, s);
    return step<__nv_bfloat16, __nv_bfloat16>(who, p, gate, s);
}

}  // extern "C"

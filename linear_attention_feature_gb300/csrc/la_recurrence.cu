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
// channels (one 128-byte row per token) and walks the sequence in rounds of
// 8 x L tokens, L consecutive ones per warp.  TMA brings a round's tiles into
// shared memory, three rounds deep.  Each thread forms the affine map (A, H) of
// its L tokens in registers, and one block barrier later applies the maps of
// the warps before it to the state that the block carries from round to round,
// walks its L tokens again from there and stores.
//
// Where there are fewer strips than the GPU holds blocks, a cluster of S blocks
// shares a strip: a round is then S x 8 x L tokens, and each block sends its map
// into the shared memory of the others (st.async, counted by an mbarrier there:
// a cluster barrier's release would wait for the round's global stores as
// well, which took half of the time).  Maps are joined in scan order, the same
// for every alignment, so repeated calls are bit-identical.
//
// Rows that TMA cannot take (strides or bases that are not multiples of 16
// bytes) are read by the threads themselves, each its own tokens and channels
// into the same places; 4-byte values with cp.async.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdio>

#include "la_internal.h"
#include "la_tc_host.h"
#include "la_tc_ptx.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 3;  // rounds of copies in flight
constexpr int kMaxCluster = 16;
constexpr long long kWaitCycles = 1LL << 32;  // bound of a wait for a copy, about 2 s

// V channels of one thread; two go through the packed fp32 instructions, which
// round like the single ones.
template <int V>
struct alignas(4 * V) Vec {
    float v[V];
};
__device__ __forceinline__ float2 f2(const Vec<2> &a) { return make_float2(a.v[0], a.v[1]); }
__device__ __forceinline__ Vec<2> vec(float2 a) { return {{a.x, a.y}}; }
template <int V>
__device__ __forceinline__ Vec<V> fma_v(Vec<V> a, Vec<V> b, Vec<V> c) {
#pragma unroll
    for (int e = 0; e < V; ++e) a.v[e] = fmaf(a.v[e], b.v[e], c.v[e]);
    return a;
}
template <int V>
__device__ __forceinline__ Vec<V> mul_v(Vec<V> a, Vec<V> b) {
#pragma unroll
    for (int e = 0; e < V; ++e) a.v[e] = __fmul_rn(a.v[e], b.v[e]);
    return a;
}
template <int V>
__device__ __forceinline__ Vec<V> add_v(Vec<V> a, Vec<V> b) {
#pragma unroll
    for (int e = 0; e < V; ++e) a.v[e] = __fadd_rn(a.v[e], b.v[e]);
    return a;
}
__device__ __forceinline__ Vec<2> fma_v(Vec<2> a, Vec<2> b, Vec<2> c) {
    return vec(__ffma2_rn(f2(a), f2(b), f2(c)));
}
__device__ __forceinline__ Vec<2> mul_v(Vec<2> a, Vec<2> b) { return vec(__fmul2_rn(f2(a), f2(b))); }
__device__ __forceinline__ Vec<2> add_v(Vec<2> a, Vec<2> b) { return vec(__fadd2_rn(f2(a), f2(b))); }
template <int V>
__device__ __forceinline__ Vec<V> all_v(float x) {
    Vec<V> r;
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = x;
    return r;
}
template <int V>
__device__ __forceinline__ Vec<V> neg_v(Vec<V> a) {
#pragma unroll
    for (int e = 0; e < V; ++e) a.v[e] = -a.v[e];
    return a;
}

// V adjacent values in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V) Mem {
    T v[V];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float &d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float x) { d = __float2bfloat16_rn(x); }
template <typename T, int V>
__device__ __forceinline__ Vec<V> widen(Mem<T, V> m) {
    Vec<V> r;
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = to_f(m.v[e]);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ Mem<T, V> narrow(Vec<V> x) {
    Mem<T, V> m;
#pragma unroll
    for (int e = 0; e < V; ++e) from_f(m.v[e], x.v[e]);
    return m;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The gate a and 1 - a, without cancellation in either.
template <int kGate, int V>
__device__ __forceinline__ void gate_of(Vec<V> z, bool need_rest, Vec<V> &a, Vec<V> &rest) {
    if (kGate == LA_GATE_VALUE) {
        a = z;
        rest = fma_v(z, all_v<V>(-1.f), all_v<V>(1.f));
    } else if (kGate == LA_GATE_LOG) {
#pragma unroll
        for (int e = 0; e < V; ++e) a.v[e] = expf(z.v[e]);
        rest = fma_v(a, all_v<V>(-1.f), all_v<V>(1.f));
        if (need_rest) {
            // 1 - e^z = -z (1 + z/2 (1 + z/3 (...))) near 0, to 2^-24 for |z| <= 1/4
            Vec<V> s = fma_v(z, all_v<V>(1.f / 720.f), all_v<V>(1.f / 120.f));
            s = fma_v(s, z, all_v<V>(1.f / 24.f));
            s = fma_v(s, z, all_v<V>(1.f / 6.f));
            s = fma_v(s, z, all_v<V>(0.5f));
            s = fma_v(s, z, all_v<V>(1.f));
            s = mul_v(s, neg_v(z));
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (fabsf(z.v[e]) <= 0.25f) rest.v[e] = s.v[e];
        }
    } else {
        // t = e^-z; the smaller of a and 1 - a first, the other as its
        // complement.  The product with log2(e) is off by 2^-24 |z| in t, but
        // a is off by only (1 - a) of that.
        const Vec<V> q = mul_v(z, all_v<V>(-1.4426950408889634f));
        Vec<V> t, r, small;
#pragma unroll
        for (int e = 0; e < V; ++e) t.v[e] = exp2_approx(q.v[e]);
        const Vec<V> d = add_v(t, all_v<V>(1.f));
#pragma unroll
        for (int e = 0; e < V; ++e) r.v[e] = rcp_approx(d.v[e]);
        const Vec<V> tr = mul_v(t, r);
#pragma unroll
        for (int e = 0; e < V; ++e) small.v[e] = z.v[e] < 0.f ? r.v[e] : tr.v[e];
        const Vec<V> other = fma_v(small, all_v<V>(-1.f), all_v<V>(1.f));
#pragma unroll
        for (int e = 0; e < V; ++e) {
            a.v[e] = z.v[e] < 0.f ? small.v[e] : other.v[e];
            rest.v[e] = z.v[e] < 0.f ? other.v[e] : small.v[e];
        }
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
    CUtensorMap map[4];  // of in, where TMA reads it
    Seq in[4];
    SeqOut out[2];
    const float *first;  // h0; backward dh_last: the carried state at the start
    float *last;         // h_last; backward dh0
    const float *h0;     // backward: h_0, for the first token's gate
    int *status;
    int B, N, C, complement, strips;
};

// Bytes of one stage: a tile [kWarps L][32 V] of the gates, then of each other
// input.
template <typename T, typename G, int V, int L, bool kBack>
constexpr int stage_bytes(int complement) {
    return kWarps * L * 32 * V *
           ((int)sizeof(G) + (int)sizeof(T) * (kBack ? 2 + complement : 1));
}

// Waits for a stage's copies or the cluster's maps, with a limit: afterwards the
// launch is marked as failed in the status word and goes on without waiting.
__device__ __forceinline__ void wait_for(uint64_t *bar, unsigned parity, bool &dead, int *status) {
    if (dead || tc::mbar_try_wait(bar, parity)) return;
    if (!tc::mbar_wait(bar, parity, clock64() + kWaitCycles, nullptr)) {
        dead = true;
        if (atomicCAS(status, 0, (int)LA_ERR_TIMEOUT) == 0)
            atomicExch(status + 1, (int)((blockIdx.x << 20) | (tc::smem_u32(bar) & 0xFFFFFu)));
    }
}

// A thread's part (A, H) of a block's map to the same place in the block `to` of
// the cluster, counted on the barrier at `bar`'s place there.
template <int V>
__device__ __forceinline__ void send_map(float *place, uint64_t *bar, int to, const Vec<V> &A,
                                         const Vec<V> &H) {
    unsigned dst, mb;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(tc::smem_u32(place)), "r"(to));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(mb) : "r"(tc::smem_u32(bar)), "r"(to));
    if constexpr (V == 2)
        asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], "
                     "{%1, %2, %3, %4}, [%5];" ::"r"(dst), "f"(A.v[0]), "f"(A.v[1]), "f"(H.v[0]),
                     "f"(H.v[1]), "r"(mb) : "memory");
    else
        asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], "
                     "{%1, %2}, [%3];" ::"r"(dst), "f"(A.v[0]), "f"(H.v[0]), "r"(mb) : "memory");
}

template <bool k>
struct Flag {
    static constexpr bool value = k;
};

template <typename T, typename G, int V, int L, int kGate, bool kTma, bool kBack>
__global__ void __launch_bounds__(kThreads, 2) rec_scan_kernel(const __grid_constant__ Params p) {
    namespace cg = cooperative_groups;
    constexpr int kTile = kWarps * L;  // tokens per block and round
    constexpr int kRow = 32 * V;
    extern __shared__ __align__(128) char stages[];
    __shared__ float warp_map[2][kWarps][2][kRow];
    __shared__ uint64_t full[kStages], maps_in[2];

    const cg::cluster_group cluster = cg::this_cluster();
    const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31;
    // the same in all lanes, so that row addresses are formed once per warp
    const int warp = __shfl_sync(~0u, tid >> 5, 0);
    const int strip = (int)(blockIdx.x / S) % p.strips, b = (int)(blockIdx.x / S) / p.strips;
    const int c0 = strip * kRow, c = c0 + lane * V;  // first channel
    const int here = min(max(p.C - c, 0), V);        // channels that exist
    const int rounds = (int)(((long long)p.N + (long long)S * kTile - 1) / ((long long)S * kTile));
    const int bytes = stage_bytes<T, G, V, L, kBack>(p.complement);

    // the cluster's maps, behind the stages: [2][S][32] of (A, H) per lane
    auto block_map = [&](int par, int k) {
        return reinterpret_cast<float *>(stages + kStages * bytes) + ((par * S + k) * 32 + lane) * 2 * V;
    };

    // A tile holds the tokens from `low` up; step j of the block in scan order
    // is its row j, or from the other end backwards.
    auto first_step = [&](int r) { return ((long long)r * S + rank) * kTile; };
    auto low = [&](int r) { return kBack ? p.N - first_step(r) - kTile : first_step(r); };
    auto row = [&](int i) { return kBack ? kTile - 1 - (warp * L + i) : warp * L + i; };
    auto tile_z = [&](int stage) { return reinterpret_cast<G *>(stages + stage * bytes); };
    auto tile_x = [&](int stage, int which) {
        return reinterpret_cast<T *>(stages + stage * bytes + kTile * kRow * (int)sizeof(G)) +
               which * kTile * kRow;
    };
    auto fetch = [&](int r) {
        const int stage = r % kStages;
        if (kTma) {
            if (tid != 0 || r >= rounds) return;
            const int t = (int)low(r);
            const uint64_t policy = tc::policy_evict_first();
            tc::mbar_arrive_expect_tx(&full[stage], bytes);
            tc::tma_load_3d(tile_z(stage), &p.map[1], &full[stage], c0, t, b, policy);
            tc::tma_load_3d(tile_x(stage, 0), &p.map[0], &full[stage], c0, t, b, policy);
            if (kBack) {
                tc::tma_load_3d(tile_x(stage, 1), &p.map[2], &full[stage], c0, t - 1, b, policy);
                if (p.complement)
                    tc::tma_load_3d(tile_x(stage, 2), &p.map[3], &full[stage], c0, t, b, policy);
            }
            return;
        }
        auto mine = [&](auto *tile, const Seq &q, int shift) {
            using E = std::remove_reference_t<decltype(*tile)>;
            const E *src = static_cast<const E *>(q.p) + b * q.b + c;
            for (int i = 0; i < L; ++i) {
                const long long t = low(r) + row(i) - shift;
                const bool ok = r < rounds && t >= 0 && t < p.N;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    E *dst = tile + row(i) * kRow + lane * V + e;
                    if (!ok || e >= here)
                        *dst = E(0.f);
                    else if (sizeof(E) == 4)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                         tc::smem_u32(dst)), "l"(src + t * q.n + e) : "memory");
                    else
                        *dst = src[t * q.n + e];
                }
            }
        };
        mine(tile_z(stage), p.in[1], 0);
        mine(tile_x(stage, 0), p.in[0], 0);
        if (kBack) {
            mine(tile_x(stage, 1), p.in[2], 1);
            if (p.complement) mine(tile_x(stage, 2), p.in[3], 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) tc::mbar_init(&full[i], 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(&maps_in[i], 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    for (int r = 0; r < kStages; ++r) fetch(r);

    Vec<V> carry = all_v<V>(0.f), h0 = all_v<V>(0.f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long at = (long long)b * p.C + c + e;
        if (p.first && e < here) carry.v[e] = p.first[at];
        if (kBack && p.h0 && e < here) h0.v[e] = p.h0[at];
    }
    bool dead = false;
    // the others' shared memory is written from here on
    if (S > 1) cluster.sync();
    for (int r = 0; r < rounds; ++r) {
        const int stage = r % kStages, par = r & 1;
        const long long s0 = first_step(r) + warp * L;  // this thread's first step
        const bool behind = s0 + L >= p.N;              // the sequence's end is in or before it
        const bool edge = behind || c0 + kRow > p.C;
        if (kTma)
            wait_for(&full[stage], (unsigned)(r / kStages) & 1u, dead, p.status);
        else
            asm volatile("cp.async.wait_group %0;" ::"n"(kBack ? kStages - 2 : kStages - 1)
                         : "memory");
        const G *zt = tile_z(stage) + lane * V;
        const T *xt = tile_x(stage, 0) + lane * V;
        // a and y (backward: a and 1 - a) of the L tokens, and their map
        Vec<V> a[L], y[L], A = all_v<V>(1.f), H = all_v<V>(0.f);
        auto form = [&](auto at_edge) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const Vec<V> z = widen<G, V>(*reinterpret_cast<const Mem<G, V> *>(zt + row(i) * kRow));
                Vec<V> x = widen<T, V>(*reinterpret_cast<const Mem<T, V> *>(xt + row(i) * kRow));
                Vec<V> rest;
                gate_of<kGate, V>(z, p.complement || kBack, a[i], rest);
                y[i] = kBack ? rest : p.complement ? mul_v(rest, x) : x;
                if (at_edge.value && s0 + i >= p.N) {
                    a[i] = all_v<V>(1.f);
                    x = y[i] = all_v<V>(0.f);
                }
                H = kBack ? mul_v(a[i], add_v(x, H)) : fma_v(a[i], H, y[i]);
                A = mul_v(A, a[i]);
            }
        };
        if (edge)
            form(Flag<true>());
        else
            form(Flag<false>());
        *reinterpret_cast<Vec<V> *>(&warp_map[par][warp][0][lane * V]) = A;
        *reinterpret_cast<Vec<V> *>(&warp_map[par][warp][1][lane * V]) = H;
        __syncthreads();
        // forward, everything of this round is in registers now; backward, the
        // round before is done with its tiles
        if (!kBack) fetch(r + kStages);
        if (kBack && r > 0) fetch(r - 1 + kStages);
        // the map of the warps before this one; the last warp joins its own to it
        // for the map of the whole block
        auto map_of = [&](int w, int which) {
            return *reinterpret_cast<const Vec<V> *>(&warp_map[par][w][which][lane * V]);
        };
        Vec<V> Ab = all_v<V>(1.f), Hb = all_v<V>(0.f), state = all_v<V>(0.f);
        for (int w = 0; w < warp; ++w) {
            const Vec<V> Aw = map_of(w, 0);
            Hb = fma_v(Aw, Hb, map_of(w, 1));
            Ab = mul_v(Ab, Aw);
        }
        if (S == 1) {
            state = fma_v(Ab, carry, Hb);
            for (int w = warp; w < kWarps; ++w) {
                const Vec<V> Aw = map_of(w, 0);
                Hb = fma_v(Aw, Hb, map_of(w, 1));
                Ab = mul_v(Ab, Aw);
            }
            carry = fma_v(Ab, carry, Hb);
        } else {
            // A block sends its map of round r + 2, to the same place, only
            // after it has those of round r + 1, and this block's goes out after
            // it has read round r's: two places are enough.
            if (tid == 0) tc::mbar_arrive_expect_tx(&maps_in[par], S * 32 * 2 * V * 4);
            if (warp == kWarps - 1) {
                const Vec<V> At = mul_v(Ab, A), Ht = fma_v(A, Hb, H);
                for (int k = 0; k < S; ++k) send_map<V>(block_map(par, rank), &maps_in[par], k, At, Ht);
            }
            wait_for(&maps_in[par], (unsigned)(r >> 1) & 1u, dead, p.status);
            for (int k = 0; k < S; ++k) {
                if (k == rank) state = fma_v(Ab, carry, Hb);
                const Vec<V> *m = reinterpret_cast<const Vec<V> *>(block_map(par, k));
                carry = fma_v(m[0], carry, m[1]);
            }
        }
        // the L tokens again, from the state that reaches them
        const long long t0 = kBack ? p.N - 1 - s0 : s0;
        auto walk = [&](auto at_edge) {
            T *o = static_cast<T *>(p.out[0].p) + b * p.out[0].b + t0 * p.out[0].n + c;
            G *oz = static_cast<G *>(p.out[1].p) + b * p.out[1].b + t0 * p.out[1].n + c;
            auto put = [&](auto *dst, const Vec<V> &v) {
                using E = std::remove_reference_t<decltype(*dst)>;
                const Mem<E, V> m = narrow<E, V>(v);
                if (kTma && (!at_edge.value || here == V)) {
                    *reinterpret_cast<Mem<E, V> *>(dst) = m;
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (e < here) dst[e] = m.v[e];
                }
            };
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const bool ok = !at_edge.value || s0 + i < p.N;
                if (!kBack) {
                    state = fma_v(a[i], state, y[i]);
                    if (ok) put(o, state);
                    o += p.out[0].n;
                    continue;
                }
                auto tile = [&](int which) {
                    return widen<T, V>(*reinterpret_cast<const Mem<T, V> *>(
                        tile_x(stage, which) + lane * V + row(i) * kRow));
                };
                Vec<V> g = tile(0), h = tile(1);
                if (at_edge.value && !ok) g = all_v<V>(0.f);
                if (at_edge.value && s0 + i == p.N - 1) h = h0;
                g = add_v(g, state);
                if (p.complement) h = fma_v(tile(2), all_v<V>(-1.f), h);
                if (ok) {
                    put(o, p.complement ? mul_v(y[i], g) : g);
                    Vec<V> dz = mul_v(g, h);
                    if (kGate != LA_GATE_VALUE) dz = mul_v(dz, a[i]);
                    if (kGate == LA_GATE_LOGIT) dz = mul_v(dz, y[i]);
                    put(oz, dz);
                }
                state = mul_v(a[i], g);
                o -= p.out[0].n;
                oz -= p.out[1].n;
            }
        };
        if (edge)
            walk(Flag<true>());
        else
            walk(Flag<false>());
        // the state behind the last token, as its warp has it: forward, these
        // are the bits that `out` was rounded from
        if (p.last && behind && s0 < p.N)
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < here) p.last[(long long)b * p.C + c + e] = state.v[e];
    }
    if (!kTma) asm volatile("cp.async.wait_all;" ::: "memory");
    if (kTma && dead)  // copies may still be under way: leave after them
        for (int r = max(0, rounds - kStages); r < rounds; ++r)
            tc::mbar_wait(&full[r % kStages], (unsigned)(r / kStages) & 1u,
                          clock64() + kWaitCycles, nullptr);
    if (S > 1) {  // no block leaves while another may still send to it
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
        asm volatile("barrier.cluster.wait;" ::: "memory");
    }
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
    auto get = [](const auto *q) {
        using E = std::remove_const_t<std::remove_reference_t<decltype(*q)>>;
        return widen<E, V>(*reinterpret_cast<const Mem<E, V> *>(q));
    };
    const Vec<V> x = get(static_cast<const T *>(p.x) + b * p.sx + c);
    const Vec<V> z = get(static_cast<const G *>(p.gates) + b * p.sg + c);
    const Vec<V> h = get(p.h + i);
    Vec<V> a, rest, s;
    gate_of<kGate, V>(z, p.complement, a, rest);
#pragma unroll
    for (int e = 0; e < V; ++e)
        s.v[e] = fmaf(a.v[e], h.v[e], p.complement ? __fmul_rn(rest.v[e], x.v[e]) : x.v[e]);
    *reinterpret_cast<Mem<float, V> *>(p.h_out + i) = narrow<float, V>(s);
    *reinterpret_cast<Mem<T, V> *>(static_cast<T *>(p.out) + b * p.so + c) = narrow<T, V>(s);
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

// Whether TMA can read the tensor: 16-byte aligned rows that do not overlap.
bool tma_ok(const Seq &q, int B, int N, int C, int elem) {
    const long long most = 1LL << 40;
    return (uintptr_t)q.p % 16 == 0 && N < 0x7fff0000 &&
           (N <= 1 || (q.n >= C && q.n * elem % 16 == 0 && q.n < most / elem)) &&
           (B <= 1 || (q.b >= C && q.b * elem % 16 == 0 && q.b < most / elem));
}

// Map of a tensor as [B][N][C], box [1][rows][columns].
bool make_map(CUtensorMap *map, const Seq &q, int B, int N, int C, int elem, int columns, int rows) {
    cudaError_t err;
    auto enc = tchost::encode_fn(&err);
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)C, (cuuint64_t)N, (cuuint64_t)B};
    const cuuint64_t any = ((cuuint64_t)C * elem + 15) / 16 * 16;  // of a dimension of one
    const cuuint64_t strides[2] = {N <= 1 ? any : (cuuint64_t)q.n * elem,
                                   B <= 1 ? any : (cuuint64_t)q.b * elem};
    const cuuint32_t box[3] = {(cuuint32_t)columns, (cuuint32_t)rows, 1}, one[3] = {1, 1, 1};
    return enc(map, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
               3, const_cast<void *>(q.p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <typename T, typename G, int V, int kGate, bool kBack>
cudaError_t launch_scan(Params &p, bool tma, cudaStream_t stream) {
    constexpr int L = kBack ? 8 : 16;
    if (tma)
        for (int i = 0; i < (kBack ? 3 + p.complement : 2); ++i)
            if (!make_map(&p.map[i], p.in[i], p.B, p.N, p.C,
                          i == 1 ? (int)sizeof(G) : (int)sizeof(T), 32 * V, kWarps * L))
                return cudaErrorInvalidValue;
    auto kern = tma ? rec_scan_kernel<T, G, V, L, kGate, true, kBack>
                    : rec_scan_kernel<T, G, V, L, kGate, false, kBack>;
    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e == cudaSuccess) p.status = device_status_word(&e);
    if (e != cudaSuccess) return e;
    p.strips = (p.C + 32 * V - 1) / (32 * V);
    const long long strips = (long long)p.B * p.strips;
    // as many blocks per strip as the GPU holds at once (two per SM) and the
    // sequence has work for
    int S = 1;
    while (S < kMaxCluster && strips * S * 2 <= 2LL * sms && (long long)S * kWarps * L < p.N)
        S *= 2;
    if (strips * S > 2147483647LL) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)kStages * stage_bytes<T, G, V, L, kBack>(p.complement) +
                        (S > 1 ? (size_t)2 * S * 32 * 2 * V * sizeof(float) : 0);
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && S > 8)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
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

template <typename T, typename G, int V, bool kBack>
cudaError_t launch_gate(Params &p, la_gate gate, bool tma, cudaStream_t s) {
    if (gate == LA_GATE_VALUE) return launch_scan<T, G, V, LA_GATE_VALUE, kBack>(p, tma, s);
    if (gate == LA_GATE_LOG) return launch_scan<T, G, V, LA_GATE_LOG, kBack>(p, tma, s);
    return launch_scan<T, G, V, LA_GATE_LOGIT, kBack>(p, tma, s);
}

template <bool kBack>
la_status launch(const char *who, Params &p, la_gate gate, la_dtype dtype, la_dtype gate_dtype,
                 cudaStream_t s) {
    // a thread takes 4 bytes of x per token: two bf16 channels
    const int v = dtype == LA_F32 ? 1 : 2;
    const int ex = dtype == LA_F32 ? 4 : 2, ez = gate_dtype == LA_F32 ? 4 : 2;
    bool tma = true;
    for (int i = 0; i < (kBack ? 3 + p.complement : 2); ++i)
        tma = tma && tma_ok(p.in[i], p.B, p.N, p.C, i == 1 ? ez : ex);
    for (int i = 0; i < 2; ++i)
        tma = tma && aligned(p.out[i].p, p.out[i].b, p.out[i].n, p.B, p.N, v, i == 1 ? ez : ex);
    using bf16 = __nv_bfloat16;
    cudaError_t e;
    if (dtype == LA_F32)
        e = launch_gate<float, float, 1, kBack>(p, gate, tma, s);
    else if (gate_dtype == LA_F32)
        e = launch_gate<bf16, float, 2, kBack>(p, gate, tma, s);
    else
        e = launch_gate<bf16, bf16, 2, kBack>(p, gate, tma, s);
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

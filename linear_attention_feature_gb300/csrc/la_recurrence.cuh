// The scan of the gated linear recurrence with a gate per channel, forward and
// backward (la_forward_recurrence, la_backward_recurrence in include/linattn.h):
//   h_t = a_t h_{t-1} + c_t x_t,   c_t = 1, or 1 - a_t with complement;
// backwards, with e_t = a_{t+1} g_{t+1} what reaches token t from later ones,
//   g_t = dout_t + e_t,  e_{t-1} = a_t g_t,
//   dx_t = c_t g_t,  dgate_t = s_t g_t (h_{t-1} - [complement] x_t),
// s_t = da_t / dgate_t.  Both directions are one affine scan per channel,
//   state <- a state + y   (forward),   state <- a (state + y)   (backward),
// walked in scan order: tokens ascending, or descending for the gradient.
//
// The data is read once.  A block takes a strip of 32 lanes x V channels (one
// 128-byte row per token) and walks the sequence in rounds of 8 x L tokens, L
// consecutive ones per warp.  TMA brings a round's tiles into shared memory some
// rounds ahead.  Each thread forms the affine map (A, H) of its L tokens in
// registers, the warps leave theirs in shared memory, and each applies those
// before it to the state that reaches the round, walks its L tokens again from
// there and stores.
//
// Two groups of 8 warps take the rounds in turn: while one waits for the state
// that reaches its round, the other works.  The last warp of a group joins the
// maps and hands the state behind its round to the other group.  Where there are
// fewer strips than SMs, a cluster of S blocks shares a strip: a round is then
// S x 8 x L tokens, and each block sends its map into the shared memory of all
// (st.async, counted by an mbarrier there: a cluster barrier's release would
// wait for the round's global stores as well, which took half of the time).
// Maps are applied in scan order, so repeated calls are bit-identical.  The grid
// is as many clusters as run at once; each takes strip after strip.
//
// Rows that TMA tiles cannot take (strides or bases that are not multiples of 16
// bytes) come by cp.async: the 16-byte units of memory that hold the strip's
// part of the row, wherever it begins in the first of them (2 x 32768 x 2047
// bf16: 273 us, against 145 us for the 2048 of whole units; when a bulk copy per
// row was tried it took 401 us against 338 us).
//
// Where even clusters would leave most SMs idle (few channels, long sequences),
// a sequence is cut into pieces and walked twice: once for the maps of the
// pieces, once from the states that they give (1 x 262144 x 64 bf16, when it was
// added: 179 us in one piece, 44 us in pieces; now 43).
//
// What bounds it (GB300, 6.78 TB/s measured copy): the latency of its instructions
// with the 16 warps that 128 registers allow, on the SMs that the strips occupy.  A
// warp spends about 660 on 16 rows of 64 bf16 channels (logistic gates with
// complement; 420 with gates as values).  A scheduler issues 0.56 a cycle (0.45),
// and no pipe is full: integer and logic 49 % (38), fp32 36 % (25), special
// functions 26 % (0), loads and stores 24 % (30); a warp's first stall is the fixed
// latency of what it just issued.  2 x 32768 x 2048 bf16 takes 145 us (5.5 TB/s) on
// the 128 SMs that 64 strips in clusters of two occupy, with gates as values 132 us
// (6.1 TB/s), with fp32 logarithms 170 us (6.3 TB/s); backward 4 x 16384 x 1024 143
// us (5.6 TB/s), 2 x 16384 x 1024 fp32 133 us (6.0 TB/s).  A warp waits as one, by a
// vote: when each lane tested for itself the forward took 152 us.  L = 16 forward
// and 8 backward: half of that doubles the share of the joining, twice needs more
// than 128 registers (32 rows with half the warps: the same time).
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cstdio>

#include "la_internal.h"
#include "la_tc.h"
#include "la_tc_host.h"
#include "la_tc_ptx.cuh"

namespace la {
namespace rec {

constexpr int kWarps = 8;        // of a group
constexpr int kGroup = 32 * kWarps;
constexpr int kThreads = 2 * kGroup;
constexpr int kMaxStages = 6;    // rounds of copies in flight, an even number
constexpr int kSlots = 4;        // rounds of maps and states kept
constexpr int kMaxCluster = 16;
constexpr int kMaxPieces = 128;  // of a sequence
constexpr int kFewStrips = 16;   // more than that are not cut into pieces
constexpr int kMaxDevices = 64;  // as device_status_word
constexpr size_t kSmem = 208 * 1024;  // stages and maps; 227 KB with the static arrays

constexpr long long kWaitCycles = 1LL << 32;  // bound of a wait, about 2 s
constexpr uint32_t kSuspendNs = 20000;  // a waiting warp sleeps this long between polls, at most
constexpr long long kFlightCycles = 1 << 20;  // a store to another block takes far less

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
// V adjacent values in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V) Mem {
    T v[V];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float &d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float x) { d = __float2bfloat16_rn(x); }
// bf16 pairs are taken apart and put together as 32-bit words: one instruction
// a value, and one a pair.
template <typename T, int V>
__device__ __forceinline__ Vec<V> widen(const Mem<T, V> *p) {
    Vec<V> r;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const unsigned u = reinterpret_cast<const unsigned *>(p)[e / 2];
            r.v[e] = __uint_as_float(u << 16);
            r.v[e + 1] = __uint_as_float(u & 0xffff0000u);
        }
    } else {
        const Mem<T, V> m = *p;
#pragma unroll
        for (int e = 0; e < V; ++e) r.v[e] = to_f(m.v[e]);
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void narrow(Mem<T, V> *p, const Vec<V> &x) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 2)
            reinterpret_cast<__nv_bfloat162 *>(p)[e / 2] = __floats2bfloat162_rn(x.v[e], x.v[e + 1]);
    } else {
        Mem<T, V> m;
#pragma unroll
        for (int e = 0; e < V; ++e) from_f(m.v[e], x.v[e]);
        *p = m;
    }
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
        if (need_rest) rest = fma_v(z, all_v<V>(-1.f), all_v<V>(1.f));
    } else if (kGate == LA_GATE_LOG) {
        // 1 - e^z = -z (1 + z/2 (1 + z/3 (...))) near 0, to 2^-24 for |z| <= 1/4; a
        // as its complement is then the nearest fp32 value, without the bias that
        // an approximate exponential adds up over a long memory
        Vec<V> s = fma_v(z, all_v<V>(1.f / 720.f), all_v<V>(1.f / 120.f));
        s = fma_v(s, z, all_v<V>(1.f / 24.f));
        s = fma_v(s, z, all_v<V>(1.f / 6.f));
        s = fma_v(s, z, all_v<V>(0.5f));
        s = fma_v(s, z, all_v<V>(1.f));
        s = mul_v(s, mul_v(z, all_v<V>(-1.f)));
        const Vec<V> near = fma_v(s, all_v<V>(-1.f), all_v<V>(1.f));
        const Vec<V> q = mul_v(z, all_v<V>(1.4426950408889634f));
        Vec<V> far;
#pragma unroll
        for (int e = 0; e < V; ++e) far.v[e] = exp2_approx(q.v[e]);
        const Vec<V> other = fma_v(far, all_v<V>(-1.f), all_v<V>(1.f));
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const bool close = fabsf(z.v[e]) <= 0.25f;
            a.v[e] = close ? near.v[e] : far.v[e];
            if (need_rest) rest.v[e] = close ? s.v[e] : other.v[e];
        }
    } else {
        // t = e^-|z|; the smaller of a and 1 - a is t / (1 + t), the other its
        // complement and so the nearest fp32 value.  The product with log2(e) is
        // off by 2^-24 |z| in t, and a by only (1 - a) of that.
        const Vec<V> q = mul_v(z, all_v<V>(1.4426950408889634f));
        Vec<V> t, r;
#pragma unroll
        for (int e = 0; e < V; ++e) t.v[e] = exp2_approx(-fabsf(q.v[e]));
        const Vec<V> d = add_v(t, all_v<V>(1.f));
#pragma unroll
        for (int e = 0; e < V; ++e) r.v[e] = rcp_approx(d.v[e]);
        const Vec<V> small = mul_v(t, r);
        const Vec<V> other = fma_v(small, all_v<V>(-1.f), all_v<V>(1.f));
#pragma unroll
        for (int e = 0; e < V; ++e) {
            a.v[e] = z.v[e] < 0.f ? small.v[e] : other.v[e];
            if (need_rest) rest.v[e] = z.v[e] < 0.f ? other.v[e] : small.v[e];
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
    long long wait_cycles;  // bound of a wait
    int hold;               // test hook: first blocks never fetch this one of the first rounds
    int B, N, C, complement, strips, stages;
    int out_vec;  // rows of the outputs are aligned to V values
    // A sequence in more than one piece of `steps` tokens (in scan order): a
    // launch with maps_only leaves the map of every piece but the last in
    // `maps`, [piece][B][C] of (A, H); the next one starts each piece from them.
    int pieces, steps, maps_only;
    float2 *maps;
    float *start;  // [B][C]: the state before the first piece, as maps_only found it
};

// Bytes of a tile's row: 32 V values, and where rows begin anywhere in a unit of
// 16 bytes, one unit more.
template <typename T, int V, bool kTma>
constexpr int row_bytes() { return 32 * V * (int)sizeof(T) + (kTma ? 0 : 16); }
// Bytes of one stage: a tile of kWarps L rows of the gates, then of each other
// input.
template <typename T, typename G, int V, int L, bool kTma, bool kBack>
constexpr int stage_bytes(int complement) {
    return kWarps * L * (row_bytes<G, V, kTma>() +
                         row_bytes<T, V, kTma>() * (kBack ? 2 + complement : 1));
}

// A warp's wait for a stage's copies, the other group's state or (kCluster) the maps
// of the cluster's blocks, with a limit: afterwards the launch is marked as failed in
// the status word, and the warp is out (false, in all lanes).
template <bool kCluster>
__device__ __forceinline__ bool wait_for(uint64_t *bar, unsigned parity, const Params &p) {
    auto done = [&]() {
        return __all_sync(~0u, kCluster ? tc::mbar_try_wait_cluster_ns(bar, parity, kSuspendNs)
                                        : tc::mbar_try_wait_ns(bar, parity, kSuspendNs));
    };
    if (done()) return true;
    const long long deadline = clock64() + p.wait_cycles;
    while (!done())
        if (__any_sync(~0u, clock64() > deadline)) {
            if (atomicCAS(p.status, 0, (int)LA_ERR_TIMEOUT) == 0)
                atomicExch(p.status + 1,
                           (int)((blockIdx.x << 20) | (tc::smem_u32(bar) & 0xFFFFFu)));
            return false;
        }
    return true;
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

// How rows are read: TMA tiles, or 16-byte units in which a row begins at a word
// or (bf16) at half a word.
enum { TILES, WORDS, HALVES };

// kComp: the input's factor is 1 (0) or 1 - a (1).
template <typename T, typename G, int V, int L, int kGate, int kComp, int kRead, bool kBack>
__global__ void __launch_bounds__(kThreads, 1) rec_scan_kernel(const __grid_constant__ Params p) {
    namespace cg = cooperative_groups;
    constexpr int kTile = kWarps * L;  // tokens per block and round
    constexpr int kRow = 32 * V;
    extern __shared__ __align__(128) char stages[];
    __shared__ __align__(16) float warp_maps[2][2][kWarps][32][2 * V];  // (A, H) per lane
    __shared__ __align__(16) float states[kSlots][32][2 * V];  // (state, product of gates)
    __shared__ uint64_t full[kMaxStages], maps_in[kSlots], state_in[kSlots];
    constexpr bool kTma = kRead == TILES;
    constexpr bool complement = kComp != 0;

    const cg::cluster_group cluster = cg::this_cluster();
    const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x % kGroup, lane = threadIdx.x & 31;
    // the same in all lanes, so that row addresses are formed once per warp
    const int group = __shfl_sync(~0u, threadIdx.x / kGroup, 0);
    const int warp = __shfl_sync(~0u, tid >> 5, 0);
    const int bytes = stage_bytes<T, G, V, L, kTma, kBack>(complement);
    const int round_steps = S * kTile;
    const int rounds = (int)(((long long)p.steps + round_steps - 1) / round_steps);  // of a piece
    const int items = p.B * p.strips * (p.pieces - p.maps_only);
    const int cid = blockIdx.x / S, clusters = gridDim.x / S;
    const int total = cid < items ? ((items - cid - 1) / clusters + 1) * rounds : 0;

    // the cluster's maps, behind the stages: [kSlots][S][32] of (A, H) per lane
    auto block_map = [&](int slot, int k) {
        return reinterpret_cast<float *>(stages + p.stages * bytes) +
               ((slot * S + k) * 32 + lane) * 2 * V;
    };

    // Item k of this cluster: a piece of a strip of a sequence.  A tile holds
    // the tokens from `low` up; step j of the block in scan order is its row j,
    // or from the other end backwards.
    struct Item {
        int b, c0, piece;
        long long begin;  // first step in scan order
        int end;          // the step after the last
    };
    auto item = [&](int k) {
        Item it;
        int i = cid + k * clusters;
        it.c0 = i % p.strips * kRow;
        i /= p.strips;
        it.b = i % p.B;
        it.piece = i / p.B;
        it.begin = (long long)it.piece * p.steps;
        it.end = (int)min(it.begin + p.steps, (long long)p.N);
        return it;
    };
    auto first_step = [&](const Item &it, int r) {
        return it.begin + (long long)r * round_steps + rank * kTile;
    };
    auto row = [&](int i) { return kBack ? kTile - 1 - (warp * L + i) : warp * L + i; };
    auto tile_z = [&](int stage) { return stages + stage * bytes; };
    auto tile_x = [&](int stage, int which) {
        return stages + stage * bytes + kTile * (row_bytes<G, V, kTma>() +
                                                 which * row_bytes<T, V, kTma>());
    };
    // round R of the cluster, round r of item `it` if there are that many, into
    // a stage; called by the threads of one group
    auto fetch = [&](int R, int stage, Item it, int r) {
        if (R >= total || (kTma && tid != 0)) return;
        if (r >= rounds) {
            it = item(R / rounds);
            r = R % rounds;
        }
        const long long s0 = first_step(it, r);
        const long long low = kBack ? p.N - s0 - kTile : s0;
        // gates, x or dout, and for a backward walk out (a token earlier) and x
        const int tensors = !kBack || p.maps_only ? 2 : complement ? 4 : 3;
        if (kTma) {
            const int t = (int)low;
            // read once, unless another launch comes for the same tiles
            const uint64_t policy = p.maps_only ? tc::policy_evict_normal() : tc::policy_evict_first();
            tc::mbar_arrive_expect_tx(
                &full[stage],
                kTile * (row_bytes<G, V, true>() + (tensors - 1) * row_bytes<T, V, true>()));
            tc::tma_load_3d(tile_z(stage), &p.map[1], &full[stage], it.c0, t, it.b, policy);
            tc::tma_load_3d(tile_x(stage, 0), &p.map[0], &full[stage], it.c0, t, it.b, policy);
            if (tensors > 2)
                tc::tma_load_3d(tile_x(stage, 1), &p.map[2], &full[stage], it.c0, t - 1, it.b, policy);
            if (tensors > 3)
                tc::tma_load_3d(tile_x(stage, 2), &p.map[3], &full[stage], it.c0, t, it.b, policy);
            return;
        }
        // the 16-byte units that hold channels [c0, c0 + kRow) of C: a thread
        // takes unit u of every kRows-th row, then each of the first threads the
        // last unit of one
        auto units = [&](auto *like, const Seq &q, int shift, char *tile) {
            using E = std::remove_pointer_t<decltype(like)>;
            constexpr int kUnits = kRow * (int)sizeof(E) / 16, kRows = kGroup / kUnits;
            const long long t0 = low - shift, line = q.n * (long long)sizeof(E);
            const int valid = min(kRow, p.C - it.c0) * (int)sizeof(E);
            const bool inside = t0 >= 0 && t0 + kTile <= p.N;
            auto one = [&](uintptr_t at, int j, int u) {
                if (16 * u < valid + (int)(at & 15) && (inside || (t0 + j >= 0 && t0 + j < p.N)))
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     tc::smem_u32(tile + j * row_bytes<E, V, false>() + 16 * u)),
                                 "l"((at & ~(uintptr_t)15) + 16 * u) : "memory");
            };
            const uintptr_t base =
                (uintptr_t)q.p + (uintptr_t)(it.b * q.b + t0 * q.n + it.c0) * sizeof(E);
            uintptr_t at = base + (uintptr_t)(tid / kUnits * line);
#pragma unroll
            for (int i = 0; i < kTile / kRows; ++i, at += (uintptr_t)(kRows * line))
                one(at, tid / kUnits + i * kRows, tid % kUnits);
            if (tid < kTile) one(base + (uintptr_t)(tid * line), tid, kUnits);
        };
        units((G *)nullptr, p.in[1], 0, tile_z(stage));
        units((T *)nullptr, p.in[0], 0, tile_x(stage, 0));
        if (tensors > 2) units((T *)nullptr, p.in[2], 1, tile_x(stage, 1));
        if (tensors > 3) units((T *)nullptr, p.in[3], 0, tile_x(stage, 2));
        // arrives when this thread's copies have
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         tc::smem_u32(&full[stage])) : "memory");
    };
    // A thread's V values of row i (in scan order, its own) of a tile.  `at` is
    // the address of the first of them in memory and `step` the bytes between
    // rows, both modulo 2^32: where the row begins in its first 16-byte unit.
    auto values = [&](auto *like, const char *tile, unsigned at, unsigned step, int i) {
        using E = std::remove_pointer_t<decltype(like)>;
        const char *line = tile + row(i) * row_bytes<E, V, kTma>() + lane * V * (int)sizeof(E);
        if constexpr (kTma) {
            return widen(reinterpret_cast<const Mem<E, V> *>(line));
        } else {
            const unsigned begin = at + i * step;
            const char *words = line + (begin & 12u);
            Vec<V> v;
            if constexpr (sizeof(E) == 4) {
#pragma unroll
                for (int e = 0; e < V; ++e) v.v[e] = *reinterpret_cast<const float *>(words + 4 * e);
            } else {  // V = 2: a pair, which may lie across two words
                unsigned u = *reinterpret_cast<const unsigned *>(words);
                if constexpr (kRead == HALVES)
                    u = __funnelshift_r(u, *reinterpret_cast<const unsigned *>(words + 4), begin * 8);
                v.v[0] = __uint_as_float(u << 16);
                v.v[V - 1] = __uint_as_float(u & 0xffff0000u);
            }
            return v;
        }
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) tc::mbar_init(&full[i], kTma ? 1 : kGroup);
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(&maps_in[i], 1);
            tc::mbar_init(&state_in[i], 32);
        }
        tc::fence_mbar_init();
    }
    __syncthreads();
    for (int i = group; i < p.stages; i += 2)
        if (i != p.hold || rank != 0) fetch(i, i, item(0), i);
    // round 0 has no state to wait for, but a phase like every other's
    if (threadIdx.x < 32) tc::mbar_arrive(&state_in[0]);
    // the others' shared memory is written from here on
    if (S > 1) cluster.sync();

    // ring positions of this group's round R, and the parities of their phases
    int stage = group, stage_phase = 0, slot = group, slot_phase = 0, turn = 0;
    int k = group / rounds, r = group % rounds;  // item and round of it
    Item it = item(0);
    int c = 0, here = 0;
    bool ends = false;  // the item ends with the sequence
    int ahead = 0;      // steps of the item from this thread's first one on
    T *o = nullptr;     // its first token in the outputs
    G *oz = nullptr;
    const long long o_turn = (kBack ? -2LL : 2LL) * round_steps * p.out[0].n;
    const long long oz_turn = -2LL * round_steps * p.out[1].n;
    // A warp that waited in vain leaves the rounds, and from there on only takes part
    // in its group's barriers: it starts no copies, sends no maps and arrives on no
    // mbarrier, so that none is counted up out of turn (a warp that goes on has seen
    // every phase before the one that it arrives for).  Who waits for it runs out of
    // time in turn.  `lost`: the first round whose barrier it has not passed.
    int lost = -1;
    for (int R = group; R < total; R += 2) {
        if (r <= 1 || turn == 0) {
            it = item(k);
            c = it.c0 + lane * V;
            here = min(max(p.C - c, 0), V);
            const long long s0 = first_step(it, r) + warp * L;  // this thread's first step
            const long long t0 = kBack ? p.N - 1 - s0 : s0;
            ahead = (int)(it.end - s0);
            ends = it.end == p.N;
            o = static_cast<T *>(p.out[0].p) + it.b * p.out[0].b + t0 * p.out[0].n + c;
            if (kBack) oz = static_cast<G *>(p.out[1].p) + it.b * p.out[1].b + t0 * p.out[1].n + c;
        }
        const bool edge = ahead <= L;  // the item ends in or before these steps
        // The state before the item's first token enters the map of the first
        // warp, and is read by that warp alone: it has been used when the state
        // behind the last token is written, which may be to the same place.
        Vec<V> init = all_v<V>(0.f), h0 = all_v<V>(0.f);
        const bool begins = r == 0 && rank == 0 && warp == 0;
        if (begins) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (p.first && e < here) init.v[e] = p.first[(long long)it.b * p.C + c + e];
            if (p.maps_only) {  // kept for the next launch, whose last piece may write there
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (it.piece == 0 && e < here) p.start[(long long)it.b * p.C + c + e] = init.v[e];
                    init.v[e] = 0.f;
                }
            }
            const int joins = p.maps_only ? 0 : it.piece;
            for (int q = 0; q < joins; q += 16) {  // 16 loads under way at once
                float2 m[16][V];
#pragma unroll
                for (int i = 0; i < 16; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        m[i][e] = q + i < joins && e < here
                                      ? p.maps[((long long)(q + i) * p.B + it.b) * p.C + c + e]
                                      : make_float2(1.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) init.v[e] = fmaf(m[i][e].x, init.v[e], m[i][e].y);
            }
        }
        if (kBack && edge && p.h0)
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < here) h0.v[e] = p.h0[(long long)it.b * p.C + c + e];
        if (!wait_for<false>(&full[stage], stage_phase, p)) {
            lost = R;
            break;
        }
        // where this thread's rows begin, see values()
        unsigned at[4] = {}, step[4] = {};
        if (!kTma)
#pragma unroll
            for (int i = 0; i < (kBack ? 4 : 2); ++i) {
                const Seq &q = p.in[i];
                const unsigned elem = i == 1 ? sizeof(G) : sizeof(T);
                const unsigned s0 = (unsigned)it.end - (unsigned)ahead;
                const unsigned t = (kBack ? (unsigned)p.N - 1u - s0 : s0) - (i == 2 ? 1u : 0u);
                step[i] = (kBack ? 0u - (unsigned)q.n : (unsigned)q.n) * elem;
                at[i] = (unsigned)(uintptr_t)q.p +
                        ((unsigned)(it.b * q.b) + t * (unsigned)q.n + (unsigned)it.c0) * elem;
            }
        const char *zt = tile_z(stage), *xt = tile_x(stage, 0);
        // a and y (backward: a and 1 - a) of the L tokens, and their map
        Vec<V> a[L], y[L], A = all_v<V>(1.f), H = all_v<V>(0.f);
        auto form = [&](auto at_edge) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const Vec<V> z = values((G *)nullptr, zt, at[1], step[1], i);
                Vec<V> x = values((T *)nullptr, xt, at[0], step[0], i);
                Vec<V> rest = all_v<V>(0.f);
                gate_of<kGate, V>(z, complement || (kBack && kGate == LA_GATE_LOGIT), a[i], rest);
                y[i] = kBack ? rest : complement ? mul_v(rest, x) : x;
                if (at_edge.value && i >= ahead) {
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
        if (begins) H = fma_v(A, init, H);
        auto maps = warp_maps[group][turn & 1];
        auto map_at = [&](float *m) { return reinterpret_cast<Vec<V> *>(m); };
        map_at(maps[warp][lane])[0] = A;
        map_at(maps[warp][lane])[1] = H;
        tc::named_bar_sync(1 + group, kGroup);
        // forward, everything of this round is in registers now; backward, the
        // group's round before is done with its tiles
        if (!kBack) fetch(R + p.stages, stage, it, r + p.stages);
        if (kBack && turn > 0)
            fetch(R - 2 + p.stages, stage >= 2 ? stage - 2 : stage - 2 + p.stages, it,
                  r - 2 + p.stages);
        // The block's map goes to all blocks of the cluster.  Four places for
        // maps: a block sends that of round R + 4 after it has all of round
        // R + 2, whose senders were past round R, the only one that reads R's.
        const bool last_warp = warp == kWarps - 1;
        if (S > 1 && last_warp) {
            Vec<V> Ab = all_v<V>(1.f), Hb = all_v<V>(0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const Vec<V> *m = map_at(maps[w][lane]);
                Hb = fma_v(m[0], Hb, m[1]);
                Ab = mul_v(Ab, m[0]);
            }
            if (lane == 0) tc::mbar_arrive_expect_tx(&maps_in[slot], S * 32 * 2 * V * 4);
            for (int to = 0; to < S; ++to)
                send_map<V>(block_map(slot, rank), &maps_in[slot], to, Ab, Hb);
        }
        // The state that reaches the round, from the other group.  Its place is
        // written again by round R + 3, after that group's barrier of round
        // R + 2, before which this round's readers are done.
        Vec<V> state = init, product = all_v<V>(1.f);
        if (!wait_for<false>(&state_in[slot], slot_phase, p)) {
            lost = R + 2;
            break;
        }
        if (r > 0) {
            state = map_at(states[slot][lane])[0];
            if (p.maps_only) product = map_at(states[slot][lane])[1];
        }
        if (S > 1 && !wait_for<true>(&maps_in[slot], slot_phase, p)) {
            lost = R + 2;
            break;
        }
        if (last_warp) {
            Vec<V> next = state;
            auto join = [&](const Vec<V> *m) {
                next = fma_v(m[0], next, m[1]);
                if (p.maps_only) product = mul_v(product, m[0]);
            };
            if (S == 1) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) join(map_at(maps[w][lane]));
            } else {
                for (int q = 0; q < S; ++q) join(map_at(block_map(slot, q)));
            }
            const int to = slot + 1 == kSlots ? 0 : slot + 1;
            map_at(states[to][lane])[0] = next;
            if (p.maps_only) {
                map_at(states[to][lane])[1] = product;
                if (r == rounds - 1 && rank == 0)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (e < here)
                            p.maps[((long long)it.piece * p.B + it.b) * p.C + c + e] =
                                make_float2(product.v[e], next.v[e]);
            }
            tc::mbar_arrive(&state_in[to]);
        }
        for (int q = 0; q < rank; ++q) {
            const Vec<V> *m = map_at(block_map(slot, q));
            state = fma_v(m[0], state, m[1]);
        }
        for (int w = 0; w < warp; ++w) {
            const Vec<V> *m = map_at(maps[w][lane]);
            state = fma_v(m[0], state, m[1]);
        }
        // the L tokens again, from there
        auto walk = [&](auto at_edge, auto whole) {
            auto put = [&](auto *dst, const Vec<V> &v) {
                using E = std::remove_reference_t<decltype(*dst)>;
                if ((kTma || p.out_vec) && (whole.value || here == V)) {
                    narrow(reinterpret_cast<Mem<E, V> *>(dst), v);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (e < here) from_f(dst[e], v.v[e]);
                }
            };
            T *to = o;
            G *toz = oz;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const bool ok = !at_edge.value || i < ahead;
                if (!kBack) {
                    state = fma_v(a[i], state, y[i]);
                    if (ok) put(to, state);
                    to += p.out[0].n;
                    continue;
                }
                Vec<V> g = values((T *)nullptr, xt, at[0], step[0], i);
                Vec<V> h = values((T *)nullptr, tile_x(stage, 1), at[2], step[2], i);
                if (at_edge.value && !ok) g = all_v<V>(0.f);
                if (at_edge.value && ends && i == ahead - 1) h = h0;
                g = add_v(g, state);
                if (complement)
                    h = fma_v(values((T *)nullptr, tile_x(stage, 2), at[3], step[3], i),
                              all_v<V>(-1.f), h);
                if (ok) {
                    put(to, complement ? mul_v(y[i], g) : g);
                    Vec<V> dz = mul_v(g, h);
                    if (kGate != LA_GATE_VALUE) dz = mul_v(dz, a[i]);
                    if (kGate == LA_GATE_LOGIT) dz = mul_v(dz, y[i]);
                    put(toz, dz);
                }
                state = mul_v(a[i], g);
                to -= p.out[0].n;
                toz -= p.out[1].n;
            }
        };
        if (!p.maps_only) {
            if (edge)
                walk(Flag<true>(), Flag<false>());
            else if (it.c0 + kRow > p.C)  // a strip that reaches beyond C
                walk(Flag<false>(), Flag<false>());
            else
                walk(Flag<false>(), Flag<true>());
            // the state behind the last token, as its warp has it: forward, these
            // are the bits that `out` was rounded from
            if (edge && p.last && ends && ahead > 0)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e < here) p.last[(long long)it.b * p.C + c + e] = state.v[e];
        }
        ahead -= 2 * round_steps;
        o += o_turn;
        if (kBack) oz += oz_turn;
        ++turn;
        if ((stage += 2) >= p.stages) stage -= p.stages, stage_phase ^= 1;
        if ((slot += 2) >= kSlots) slot -= kSlots, slot_phase ^= 1;
        for (r += 2; r >= rounds; r -= rounds) ++k;
    }
    if (!kTma) asm volatile("cp.async.wait_all;" ::: "memory");
    if (lost >= 0) {
        for (int R = lost; R < total; R += 2) tc::named_bar_sync(1 + group, kGroup);
        // the tiles that this thread asked for and has not waited for: the last of
        // each stage, the latest with round lost - 2, or before the rounds
        if (kTma && tid == 0)
            for (int left = p.stages, i = lost - 2 + left - (kBack && lost > group ? 2 : 0);
                 left > 0; left -= 2, i -= 2)
                if (i >= 0 && i < total && !(i == p.hold && rank == 0))
                    tc::mbar_wait(&full[i % p.stages], (unsigned)(i / p.stages) & 1u,
                                  clock64() + kWaitCycles, nullptr);
    }
    if (S > 1) {  // no block leaves while another may still send to it
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
        asm volatile("barrier.cluster.wait;" ::: "memory");
        // blocks that went on for longer have sent maps that nobody counts here
        if (lost >= 0)
            for (const long long until = clock64() + kFlightCycles; clock64() < until;)
                __nanosleep(1000);
    }
}

inline la_status rec_fail(la_status s, const char *who, const char *msg) {
    char text[200];
    std::snprintf(text, sizeof(text), "%s: %s", who, msg);
    set_last_error(text);
    return s;
}

inline bool aligned(const void *p, long long b, long long n, int B, int N, int v, int elem) {
    return (uintptr_t)p % (uintptr_t)(v * elem) == 0 && (B <= 1 || b % v == 0) &&
           (N <= 1 || n % v == 0);
}

// Whether TMA can read the tensor: 16-byte aligned rows that do not overlap.
inline bool tma_ok(const Seq &q, int B, int N, int C, int elem) {
    const long long most = 1LL << 40;
    return (uintptr_t)q.p % 16 == 0 && N < 0x7fff0000 &&
           (N <= 1 || (q.n >= C && q.n * elem % 16 == 0 && q.n < most / elem)) &&
           (B <= 1 || (q.b >= C && q.b * elem % 16 == 0 && q.b < most / elem));
}

// Map of a tensor as [B][N][C], box [1][rows][columns].
inline bool make_map(CUtensorMap *map, const Seq &q, int B, int N, int C, int elem, int columns, int rows) {
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

// How a call is cut: clusters of S blocks, pieces of a sequence.
struct Cut {
    int S, clusters, pieces, steps, stages;
    size_t smem;
};

// The cheapest cut, counted in rounds of a block alone (about 1.1 us forward, 0.95
// us backward for bf16 logits with complement): a cluster takes ceil(items /
// clusters) strips, one after the other, each of ceil(steps / (S tile)) rounds and
// about two more for the start.  Measured, a round of S blocks takes 1.2 to 1.3
// times one of a block at S = 16 (more maps to join).  clusters_of: how many run
// at once.
template <bool kBack, typename F>
Cut best_cut(const Params &p, int tile, int bytes, int V, int least_stages, F &&clusters_of) {
    const long long items = (long long)p.B * p.strips;
    Cut best{};
    double cost = 0;
    auto stages_of = [&](int S, size_t &smem) {
        const size_t maps = (size_t)kSlots * S * 32 * 2 * V * sizeof(float);
        const int stages = std::min<int>(kMaxStages, (int)((kSmem - maps) / bytes) / 2 * 2);
        smem = (size_t)stages * bytes + maps;
        return stages;
    };
    for (int S = 1; S <= kMaxCluster; ++S) {
        if (S > 1 && (long long)(S - 1) * tile >= p.N) break;
        size_t smem;
        const int stages = stages_of(S, smem);
        if (stages < least_stages) break;
        const long long most = clusters_of(S, smem);
        if (most < 1) continue;
        const long long waves = (items + most - 1) / most;
        const long long rounds = ((long long)p.N + (long long)S * tile - 1) / ((long long)S * tile);
        const double c = (double)waves * ((1 + 0.015 * S) * (double)rounds + 2) + 5;
        if (!best.S || c < cost) {
            cost = c;
            best = {S, (int)std::min(items, most), 1, p.N, stages, smem};
        }
    }
    // In pieces, of blocks alone: a round of the maps takes 0.82 of one of the walk
    // forward (of its three tensors two are read), 0.55 backward; two launches, the
    // maps between them and the joining took 10 rounds more.  1 x N x C bf16, in
    // clusters / in pieces, when the weights were fitted: forward 65536 x 256 49 / 38 us, x 384 50 / 57; backward
    // 65536 x 512 109 / 95, x 768 129 / 139; 16384 x 512 32 / 30, 8192 x 512 19 / 20.
    if (!best.S || items > kFewStrips) return best;
    size_t smem;
    const int stages = stages_of(1, smem);
    const long long most = clusters_of(1, smem);
    for (int P = 2; P <= kMaxPieces; ++P) {
        const int steps = (int)(((long long)p.N + (long long)P * tile - 1) / ((long long)P * tile)) * tile;
        const int pieces = (int)(((long long)p.N + steps - 1) / steps);
        if (pieces != P || steps < 4 * tile) continue;
        const double rounds = steps / tile + 2;
        const double c =
            (kBack ? 0.55 : 0.82) * rounds * (double)((items * (P - 1) + most - 1) / most) +
            rounds * (double)((items * P + most - 1) / most) + 10;
        if (c < cost) {
            cost = c;
            best = {1, (int)std::min(items * P, most), P, steps, stages, smem};
        }
    }
    return best;
}

struct Workspace {
    void *p;
    size_t bytes;
};

template <typename T, typename G, int V, int kGate, int kComp, bool kBack>
la_status launch_scan(const char *who, Params &p, int read, Workspace ws, cudaStream_t stream) {
    const bool tma = read == TILES;
    constexpr int L = kBack ? 8 : 16, kTile = kWarps * L;
    auto cuda = [&](cudaError_t e) { return rec_fail(LA_ERR_CUDA, who, cudaGetErrorString(e)); };
    if (tma)
        for (int i = 0; i < (kBack ? 3 + p.complement : 2); ++i)
            if (!make_map(&p.map[i], p.in[i], p.B, p.N, p.C,
                          i == 1 ? (int)sizeof(G) : (int)sizeof(T), 32 * V, kTile))
                return rec_fail(LA_ERR_CUDA, who, "tensor map");
    auto kern = rec_scan_kernel<T, G, V, L, kGate, kComp, TILES, kBack>;
    if (read == WORDS) kern = rec_scan_kernel<T, G, V, L, kGate, kComp, WORDS, kBack>;
    if constexpr (sizeof(T) == 2)
        if (read == HALVES) kern = rec_scan_kernel<T, G, V, L, kGate, kComp, HALVES, kBack>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) p.status = device_status_word(&e);  // also bounds dev
    if (e != cudaSuccess) return cuda(e);
    // clusters that run at once (one block per SM whatever the stages), looked up
    // once; 0: not yet, -1: none
    static std::atomic<int> known[kMaxDevices][3][kMaxCluster + 1];
    std::atomic<int> *at_once = known[dev][read];
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (at_once[1].load() == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda(e);
        for (int S = kMaxCluster; S >= 1; --S) {
            int got = 0;
            cfg.gridDim = dim3((unsigned)S);
            cfg.dynamicSmemBytes = kSmem;
            at[0].val.clusterDim = {(unsigned)S, 1, 1};
            if (cudaOccupancyMaxActiveClusters(&got, kern, &cfg) != cudaSuccess)
                (void)cudaGetLastError();
            at_once[S].store(got > 0 ? got : -1);
        }
    }
    p.strips = (p.C + 32 * V - 1) / (32 * V);
    const int bytes = tma ? stage_bytes<T, G, V, L, true, kBack>(p.complement)
                          : stage_bytes<T, G, V, L, false, kBack>(p.complement);
    // backward, a stage is refilled two rounds after its own
    const Cut cut = best_cut<kBack>(p, kTile, bytes, V, kBack ? 4 : 2,
                             [&](int S, size_t) { return at_once[S].load(); });
    if (!cut.S) return rec_fail(LA_ERR_UNSUPPORTED, who, "no kernel configuration fits");
    p.stages = cut.stages;
    p.pieces = cut.pieces;
    p.steps = cut.steps;
    void *mine = nullptr;
    if (cut.pieces > 1) {
        const size_t states = (size_t)p.B * p.C;
        const size_t need = (sizeof(float2) * (cut.pieces - 1) + sizeof(float)) * states;
        if (ws.p) {
            if (ws.bytes < need || (uintptr_t)ws.p % 16)
                return rec_fail(LA_ERR_INVALID_ARG, who, "workspace too small or not 16-byte aligned");
            p.maps = static_cast<float2 *>(ws.p);
        } else {
            e = tc_workspace_alloc(&mine, need, stream);
            if (e != cudaSuccess) {
                (void)cudaGetLastError();
                return rec_fail(LA_ERR_NO_MEMORY, who, "workspace allocation");
            }
            p.maps = static_cast<float2 *>(mine);
        }
        p.start = reinterpret_cast<float *>(p.maps + (cut.pieces - 1) * states);
    }
    p.wait_cycles = kWaitCycles;
    p.hold = -1;
    tc_debug_take_timeout(&p.wait_cycles, &p.hold);
    cfg.dynamicSmemBytes = cut.smem;
    at[0].val.clusterDim = {(unsigned)cut.S, 1, 1};
    int launches = 0;
    for (int pass = cut.pieces > 1 ? 0 : 1; pass < 2 && e == cudaSuccess; ++pass) {
        p.maps_only = pass == 0;
        const int items = p.B * p.strips * (cut.pieces - p.maps_only);
        cfg.gridDim = dim3((unsigned)(std::min(cut.clusters, items) * cut.S));
        e = cudaLaunchKernelEx(&cfg, kern, p);
        launches += e == cudaSuccess;
        p.first = p.start;  // of the second pass
    }
    note_launches(launches);
    if (mine) {
        const cudaError_t ef = cudaFreeAsync(mine, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e == cudaSuccess ? LA_OK : cuda(e);
}

template <typename T, typename G, int V, int kGate, bool kBack>
la_status launch_comp(const char *who, Params &p, int read, Workspace ws, cudaStream_t s) {
    return p.complement ? launch_scan<T, G, V, kGate, 1, kBack>(who, p, read, ws, s)
                        : launch_scan<T, G, V, kGate, 0, kBack>(who, p, read, ws, s);
}

template <typename T, typename G, int V, bool kBack>
la_status launch_gate(const char *who, Params &p, la_gate gate, int read, Workspace ws,
                      cudaStream_t s) {
    if (gate == LA_GATE_VALUE)
        return launch_comp<T, G, V, LA_GATE_VALUE, kBack>(who, p, read, ws, s);
    if (gate == LA_GATE_LOG) return launch_comp<T, G, V, LA_GATE_LOG, kBack>(who, p, read, ws, s);
    return launch_comp<T, G, V, LA_GATE_LOGIT, kBack>(who, p, read, ws, s);
}

template <bool kBack>
la_status launch(const char *who, Params &p, la_gate gate, la_dtype dtype, la_dtype gate_dtype,
                 Workspace ws, cudaStream_t s) {
    if (p.B * ((p.C + 31LL) / 32) > 2147483647LL / kMaxPieces)
        return rec_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
    // a thread takes 4 bytes of x per token: two bf16 channels
    const int v = dtype == LA_F32 ? 1 : 2;
    const int ex = dtype == LA_F32 ? 4 : 2, ez = gate_dtype == LA_F32 ? 4 : 2;
    bool tma = true, words = true;
    for (int i = 0; i < (kBack ? 3 + p.complement : 2); ++i) {
        const int elem = i == 1 ? ez : ex;
        tma = tma && tma_ok(p.in[i], p.B, p.N, p.C, elem);
        words = words && aligned(p.in[i].p, p.in[i].b, p.in[i].n, p.B, p.N, 4 / elem, elem);
    }
    p.out_vec = 1;
    for (int i = 0; i < 2; ++i)
        p.out_vec = p.out_vec && aligned(p.out[i].p, p.out[i].b, p.out[i].n, p.B, p.N, v,
                                         i == 1 ? ez : ex);
    const int read = tma && p.out_vec ? TILES : words ? WORDS : HALVES;
    using bf16 = __nv_bfloat16;
    if (dtype == LA_F32) return launch_gate<float, float, 1, kBack>(who, p, gate, read, ws, s);
    if (gate_dtype == LA_F32) return launch_gate<bf16, float, 2, kBack>(who, p, gate, read, ws, s);
    return launch_gate<bf16, bf16, 2, kBack>(who, p, gate, read, ws, s);
}

}  // namespace rec
}  // namespace la

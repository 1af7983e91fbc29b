// Linear cross attention on tcgen05 tensor cores (bf16, head sizes up to 128 that are
// multiples of 8, rows on 16-byte boundaries); the formulas are in la_cross.cu.
//
// Four persistent kernels, one block per SM, each over an equal piece of one list of
// tiles of tokens (for each sequence and head of keys), whatever the sequences'
// lengths:
//   state   S, z of the keys:        [S | z] = phi(K)^T [V | 1]
//   read    outputs:                 [y den | den] = phi(Q) [S | z]
//   qgrad   dq, and sums dS, dz:     [G | .] = dY S'^T, [dS | -dz] = psi^T [dY | t]
//   kgrad   dk and dv:               dphi(K) = V dS^T + dz, dV = phi(K) dS
// All of them are bound by reading and writing the tokens once; the products run
// beside that.  A state whose tokens lie in several pieces is left in parts, which
// join_kernel adds in order.
//
// What is rounded to bf16, and why that is enough:
//   state   phi(k) is kept as two bf16 numbers, high and low (2^-16 of it), since S and
//           z are results in fp32; V is exact.  The tensor cores cut off what they add,
//           so a product's sum ends after 256 tokens and is added to the ones before,
//           rounded, by the computing warps.  (That running sum is in TMEM, too: held in
//           registers it made phi spill, 60 us instead of 52 for 4 x 8 x 16384 x 128.)
//   read    phi(q) and S as one each, z as two: 2^-8 of a weighted mean's terms, as
//           much as y's own rounding.
//   qgrad   r (S dy - t z) is the same for S' = S - z m^T, any m.  With m = S^T z / z.z,
//           the mean of the values as z weighs it, S' has none of the large common part
//           that cancels, and one bf16 number is enough.  psi = r phi(q) as one; the
//           sums of psi and of psi t then go by the same rounded psi, t as two.  A
//           product's sum ends after 2048 tokens; the sums are added in fp32.
//   kgrad   dS as two for dphi(K), where dS v and dz cancel for values with a mean far
//           from 0; as one for dV.
//
// Roles (608 threads): warp 0 fetches tiles (TMA), warp 1 issues products, warps 2-17
// take phi, empty TMEM and compute what lies between, warp 18 stores tiles (TMA).  The
// computing warps set the pace: with 8 of them, and phi with a branch, the kernels were
// bound by latency and instructions at a third of the memory's rate.  They do not fill a
// pipe now (0.36 to 0.62 instructions issued per cycle, tensor cores 9 to 21 %, memory
// 48 to 54 %): what is left is the way of a tile through fetch, phi, product and emptying,
// of which two to four are under way in shared memory, and some 8 us of start and end.
#include <cuda_bf16.h>

#include <algorithm>

#include "la_cross.h"
#include "la_layer.cuh"
#include "la_tc.h"
#include "la_tc_common.cuh"
#include "la_tc_host.h"
#include "la_tc_ptx.cuh"

namespace la {
namespace cross {
namespace {

using namespace la::tc;
using namespace la::tcc;

constexpr int kThreads = 608, kC0 = 64, kC = 512;  // all; the computing ones: from, number
constexpr int kWarpsC = kC / 32, kParts = kWarpsC / 4;  // warps that share rows of TMEM
// Where tiles are independent, two groups of computing warps take them in turn, so that
// one works while the other waits.
constexpr int kG = kC / 2, kWarpsG = kG / 32;
constexpr int BAR_C = 1;
constexpr uint32_t kTmemCols = 512;  // all: one block per SM (d <= 64 would do with half)

struct Params {
    int B, Hk, G, L, d, phi, norm;  // L: tokens of a head
    const int *lengths;             // keys' side, or NULL
    const float *S, *z;             // read, qgrad, kgrad (there dS, dz)
    float *So, *zo;                 // state, qgrad: whole states
    float *part;                    // and parts, [blocks][2][d d + d]
    int4 *info;                     // of each block: the state that its first part
                                    // continues (-1: none), first and last block of it
    float zsign;
    int *status;
    long long timeout;  // clock cycles per wait
    int hold;           // test hook: a block fetches no tile from this one of its own on, or -1
};

__device__ __forceinline__ int tokens_of(const Params &p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
}

// A place in the list: tile of head `seg` of sequence b, which has `len` tokens.  F:
// tiles of a head of so many tokens.
template <typename F>
struct Walk {
    F count;
    const Params &p;
    int segs, b, seg, tile, tiles, len;

    __device__ __forceinline__ Walk(F f, const Params &p, const Piece &x)
        : count(f), p(p), segs(p.Hk), b(x.b), seg(0), tile(0), tiles(1), len(0) {
        if (x.x0 < x.x1) {
            len = tokens_of(p, b);
            tiles = count(len);
            seg = (int)(x.rest <= 0x7fffffff ? (unsigned)x.rest / (unsigned)tiles : x.rest / tiles);
            tile = (int)(x.rest - (long long)seg * tiles);
        }
    }
    __device__ __forceinline__ bool last() const { return tile == tiles - 1; }
    __device__ __forceinline__ void next() {
        if (++tile < tiles) return;
        tile = 0;
        if (++seg < segs) return;
        seg = 0;
        do {
            if (++b >= p.B) return;
            len = tokens_of(p, b);
            tiles = count(len);
        } while (tiles == 0);
    }
};
template <typename F>
__device__ __forceinline__ Walk<F> walk(F f, const Params &p, const Piece &x) {
    return Walk<F>(f, p, x);
}

// Whether a block's tile j may be fetched into a stage, once `empty` says that it is free.
// Where a wait has given up that may be untrue: it passes, and with it what follows, while
// the stage's copy is under way, whose barrier must not be armed a second time.
__device__ __forceinline__ bool may_fetch(const Params &p, uint64_t *empty, uint32_t parity, int j,
                                          const Ctx &cx) {
    return j != p.hold && wait_bar(empty, parity, cx) && !*cx.abort;
}

// ------------------------------------------------------------------ TMA, 4-D maps

__device__ __forceinline__ void load_tile(void *dst, const CUtensorMap *map, uint64_t *bar, int c,
                                          int tok, int h, int b, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c), "r"(tok), "r"(h), "r"(b), "r"(smem_u32(bar)), "l"(policy) : "memory");
}
__device__ __forceinline__ void store_tile(const CUtensorMap *map, const void *src, int c, int tok,
                                           int h, int b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::
            "l"(map), "r"(smem_u32(src)), "r"(c), "r"(tok), "r"(h), "r"(b) : "memory");
}

// ------------------------------------------------------------------ tiles

// Bytes from a tile's start to feature `col` (a multiple of 8) of row `row`; a tile has
// an atom of 64 features after the other, `rows` rows each.
__device__ __forceinline__ uint32_t tile_at(int rows, int row, int col) {
    return (uint32_t)(col >> 6) * (uint32_t)rows * 128u + sw128_offset(row, col & 63);
}

__device__ __forceinline__ void open8(const uint4 x, float (&e)[8]) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e[2 * i] = __uint_as_float(u[i] << 16);
        e[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 shut8(const float (&e)[8]) {
    return make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                      pack_bf16x2(e[6], e[7]));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max(x, 0), and NaN of NaN.
__device__ __forceinline__ float above(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}
// elu(x) + 1 = max(x, 0) + exp(min(x, 0)), of pairs.
__device__ __forceinline__ float2 exp_below(float2 x) {
    const float2 u = __fmul2_rn(make_float2(fminf(x.x, 0.f), fminf(x.y, 0.f)),
                                make_float2(1.44269504088896341f, 1.44269504088896341f));
    return make_float2(exp2_fast(u.x), exp2_fast(u.y));
}
__device__ __forceinline__ void phi8(float (&e)[8], int phi) {
    if (!phi) return;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 x = make_float2(e[i], e[i + 1]);
        const float2 f = __fadd2_rn(make_float2(above(x.x), above(x.y)), exp_below(x));
        e[i] = f.x;
        e[i + 1] = f.y;
    }
}
// phi' from phi: where x > 0, phi > 1 and the slope is 1; elsewhere it is phi itself.
__device__ __forceinline__ float slope_of_phi(float f, int phi) {
    return !phi ? 1.f : fminf(f, 1.f);
}
// What eight numbers lose as bf16, as bf16.  Of an infinity that is the same infinity (less
// the largest number below it), so that the two parts have a sum.  (The bounds cost the
// states' kernel 2 %; a look at the keys' largest instead costs as much.)
__device__ __forceinline__ uint4 low8(const float (&e)[8], const uint4 high) {
    const auto bound = [](uint32_t u) { return bf2_max(bf2_min(u, 0x7F7F7F7Fu), 0xFF7FFF7Fu); };
    float h[8];
    open8(make_uint4(bound(high.x), bound(high.y), bound(high.z), bound(high.w)), h);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 l = __fadd2_rn(make_float2(e[i], e[i + 1]), make_float2(-h[i], -h[i + 1]));
        h[i] = l.x;
        h[i + 1] = l.y;
    }
    return shut8(h);
}
// A number as a pair of bf16, high and low; the low one of an infinity is 0.
__device__ __forceinline__ uint32_t split(float x) {
    const float high = __bfloat162float(__float2bfloat16_rn(x));
    return pack_bf16x2(x, fabsf(high) < INFINITY ? x - high : 0.f);
}

__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void sync_compute() { named_bar_sync(BAR_C, kC); }

// Set-up that all kernels share: barriers are initialised by `init` (one thread), TMEM is
// taken, the dependency on the kernel before is waited for.
template <typename F>
__device__ __forceinline__ uint32_t begin(uint32_t *tmem_base, F init) {
    grid_dep_launch();
    if (threadIdx.x == 0) {
        init();
        fence_mbar_init();
    }
    if (threadIdx.x >> 5 == 1) {
        tmem_alloc(tmem_base, kTmemCols);
        tmem_relinquish();
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dep_wait();
    return *tmem_base;
}
__device__ __forceinline__ void end(uint32_t tmem) {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x >> 5 == 1) tmem_dealloc(tmem, kTmemCols);
}

__device__ __forceinline__ void clear(uint8_t *at, int bytes) {
    for (int i = threadIdx.x; i < bytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(at)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Where a computing thread's results lie in TMEM: lane (row of the product) and part of
// the columns.
struct Mine {
    int et, row, part, group;
    uint32_t lane_base;
    __device__ __forceinline__ explicit Mine(uint32_t tmem) {
        et = threadIdx.x - kC0;
        const int quarter = (threadIdx.x >> 5) & 3;
        row = quarter * 32 + (threadIdx.x & 31);
        part = et / (kC / kParts);
        group = et / kG;
        lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    }
};

// N consecutive columns of this thread's lane, as fp32, after the wait.
__device__ __forceinline__ void tmem_get(uint32_t at, uint32_t (&v)[32]) {
    tmem_ld32(at, v);
    tmem_wait_ld();
    reg_fence(v);
}
__device__ __forceinline__ void tmem_get(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
    tmem_wait_ld();
    reg_fence(r);
}

__device__ __forceinline__ void tmem_put(uint32_t at, const uint32_t (&v)[32]) { tmem_st32(at, v); }
__device__ __forceinline__ void tmem_put(uint32_t at, const uint32_t (&v)[16]) { tmem_st16(at, v); }

// The sums of one state, of which a computing thread has kCols columns of row a, and
// z[a] (part 0).  In TMEM the product's columns from kSplit on lie 16 further on, behind
// z's, of which there are kZ.
template <int DK, int kSplit, int kZ>
struct Sums {
    static constexpr int kCols = DK / kParts;
    static __device__ __forceinline__ void get(const Mine &me, uint32_t base, uint32_t (&v)[kCols],
                                               float &z) {
        const int c = me.part * kCols;
        tmem_get(me.lane_base + base + c + (c < kSplit ? 0 : 16), v);
        if (me.part > 0) return;
        uint32_t v0 = tmem_ld1(me.lane_base + base + kSplit), v1 = 0;
        if (kZ == 2) v1 = tmem_ld1(me.lane_base + base + kSplit + 1);
        tmem_wait_ld();
        reg_fence(v0);
        reg_fence(v1);
        z = kZ == 2 ? u2f(v0) + u2f(v1) : u2f(v0);
    }
    // To the state itself, or to part `slot` (>= 0) of this block; `more`: added to what this
    // thread wrote there before (nobody else adds to it, so the order is fixed).
    static __device__ __forceinline__ void write(const Params &p, const Mine &me, long long state,
                                                 int slot, const uint32_t (&v)[kCols], float z,
                                                 bool more = false) {
        const int a = me.row, c0 = me.part * kCols;
        if (a >= p.d) return;
        const long long dd = (long long)p.d * p.d;
        float *S, *z_to;
        if (slot < 0) {
            S = p.So + state * dd;
            z_to = p.zo + state * p.d;
        } else {
            S = p.part + (2 * (long long)blockIdx.x + slot) * (dd + p.d);
            z_to = S + dd;
        }
        S += (long long)a * p.d + c0;
#pragma unroll
        for (int e = 0; e < kCols; e += 4)
            if (c0 + e < p.d) {
                const float4 u = make_float4(u2f(v[e]), u2f(v[e + 1]), u2f(v[e + 2]), u2f(v[e + 3]));
                if (more)
                    atomicAdd(reinterpret_cast<float4 *>(S + e), u);
                else
                    *reinterpret_cast<float4 *>(S + e) = u;
            }
        if (me.part > 0) return;
        if (more)
            atomicAdd(z_to + a, p.zsign * z);
        else
            z_to[a] = p.zsign * z;
    }
};

// A state S in registers, 8 numbers at a time: number i of a computing thread is row
// (et + 512 i) / (DK / 8), columns (et + 512 i) % (DK / 8) 8 on.  All loads are under way
// at once.
template <int DK>
struct Loaded {
    static constexpr int kN = DK * DK / 8 / kC;
    float4 u[kN], v[kN];
    static __device__ __forceinline__ int row(int et, int i) { return (et + kC * i) / (DK / 8); }
    static __device__ __forceinline__ int col(int et, int i) {
        return (et + kC * i) % (DK / 8) * 8;
    }
    __device__ __forceinline__ void load(const float *S, int d, int et) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int a = row(et, i), c = col(et, i);
            u[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (a < d && c < d) {
                const float4 *s4 = reinterpret_cast<const float4 *>(S + (long long)a * d + c);
                u[i] = __ldcg(s4);
                v[i] = __ldcg(s4 + 1);
            }
        }
    }
    __device__ __forceinline__ void get(int i, float (&e)[8]) const {
        e[0] = u[i].x, e[1] = u[i].y, e[2] = u[i].z, e[3] = u[i].w;
        e[4] = v[i].x, e[5] = v[i].y, e[6] = v[i].z, e[7] = v[i].w;
    }
};

// ------------------------------------------------------------------ state
//
// phi(K) as high and low, high in K's place, low in a ring of its own; both times [V | 1]
// into TMEM, DK rows a, DK + 16 columns.  4 x 8 x 16384 x 128 (ragged, 198 MB read): 53 us,
// 3.7 TB/s; without phi and products it is 42 us.  Tiles of 64 tokens, since four stages of
// them fit with d = 128 (32 tokens: 63 us).  Fetching tiles into L2 ahead, 59 us.

template <int DK>
struct StateLayout {
    static constexpr int TOK = DK == 128 ? 64 : 128, KB = DK / 64;
    // A stage: K, V and behind V the column of ones, one operand of DK + 16 columns.
    static constexpr int ATOM = TOK * 128, TILE = KB * ATOM, STAGE = 2 * TILE + ATOM;
    static constexpr int STAGES = DK == 128 ? 4 : 3, LOWS = 3;
    static constexpr int OFF_LOW = STAGES * STAGE, OFF_SMALL = OFF_LOW + LOWS * TILE;
    static constexpr int GROUP = 256 / TOK;  // tiles between two emptyings
};
struct StateSmall {
    uint64_t full[4], empty[4], ready[4], low_empty[3], acc_full[2], acc_empty[2], fin;
    long long plan[kThreads / 32 + 2];
    uint32_t tmem;
    int abort;
};

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
state_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
             const Params p) {
    using L = StateLayout<DK>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                ~uintptr_t(1023));
    StateSmall &sm = *reinterpret_cast<StateSmall *>(smem + L::OFF_SMALL);
    for (int i = 0; i < L::STAGES; ++i) clear(smem + i * L::STAGE + 2 * L::TILE, L::ATOM);
    __syncthreads();
    for (int i = threadIdx.x; i < L::STAGES * L::TOK; i += kThreads)
        *reinterpret_cast<uint16_t *>(smem + i / L::TOK * L::STAGE + 2 * L::TILE +
                                      sw128_offset(i % L::TOK, 0)) =
            (uint16_t)(kBf16One2 & 0xFFFFu);
    const uint32_t tmem = begin(&sm.tmem, [&] {
        sm.abort = 0;
        for (int i = 0; i < L::STAGES; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
            mbar_init(&sm.ready[i], kWarpsG);
        }
        for (int i = 0; i < L::LOWS; ++i) mbar_init(&sm.low_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], kWarpsC);
        }
        mbar_init(&sm.fin, 1);
    });
    const Ctx cx{&sm.abort, p.status, p.timeout};
    auto count = [](int len) { return max(1, (len + L::TOK - 1) / L::TOK); };
    const Piece x = find_piece<kThreads>(
        p.B, p.Hk, 4, [&](int b) { return count(tokens_of(p, b)); }, sm.plan);
    const int steps = (int)(x.x1 - x.x0);
    if (threadIdx.x == 0) p.info[blockIdx.x] = make_int4(-1, 0, 0, 0);
    auto w = walk(count, p, x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_first();
            int j = 0;
            for (; j < steps; ++j, w.next()) {
                const int st = j % L::STAGES;
                if (!may_fetch(p, &sm.empty[st], ((j / L::STAGES) & 1) ^ 1, j, cx)) break;
                uint8_t *at = smem + st * L::STAGE;
                mbar_arrive_expect_tx(&sm.full[st], 2 * L::TILE);
                for (int a = 0; a < L::KB; ++a) {
                    load_tile(at + a * L::ATOM, &tk, &sm.full[st], 64 * a, w.tile * L::TOK, w.seg,
                              w.b, pol);
                    load_tile(at + L::TILE + a * L::ATOM, &tv, &sm.full[st], 64 * a,
                              w.tile * L::TOK, w.seg, w.b, pol);
                }
            }
            for (int i = max(0, j - L::STAGES); i < j; ++i)  // all have landed
                settle_wait(&sm.full[i % L::STAGES], (i / L::STAGES) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t id = idesc_bf16(128, DK + 16, 1, 1);
            constexpr uint32_t lboA = DK == 128 ? L::ATOM : 0;  // DK = 64: rows 64.. repeat
            int g = 0, in = 0;
            for (int j = 0; j < steps; ++j, w.next()) {
                const int st = j % L::STAGES;
                if (in == 0) wait_bar_spin(&sm.acc_empty[g & 1], ((g >> 1) & 1) ^ 1, cx);
                wait_bar_spin(&sm.ready[st], (j / L::STAGES) & 1, cx);
                tc_fence_after();
                const uint32_t hi = smem_u32(smem + st * L::STAGE), vb = hi + L::TILE;
                const uint32_t lo = smem_u32(smem + L::OFF_LOW + j % L::LOWS * L::TILE);
                const uint32_t acc = tmem + (g & 1) * 160;
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < L::TOK / 16; ++ks) {
                        const uint64_t a = sdesc_sw128((part ? lo : hi) + ks * 2048, lboA, 1024);
                        mma_ss(acc, a, sdesc_sw128(vb + ks * 2048, L::ATOM, 1024), id,
                               in > 0 || part > 0 || ks > 0);
                    }
                mma_commit(&sm.empty[st]);
                mma_commit(&sm.low_empty[j % L::LOWS]);
                if (++in == L::GROUP || w.last() || j == steps - 1) {
                    mma_commit(&sm.acc_full[g & 1]);
                    ++g;
                    in = 0;
                }
            }
            mma_commit(&sm.fin);
            settle_wait(&sm.fin, 0);
        }
    } else if (warp < 2 + kWarpsC) {
        const Mine me(tmem);
        constexpr int kChunks = DK / 8 / (kG / L::TOK);
        const int row = me.et % L::TOK, part = me.et % kG / L::TOK;
        using Sum = Sums<DK, DK, 1>;
        constexpr uint32_t kTotal = 320;  // TMEM column of the running sum
        int g = 0, in = 0, first = w.tile;
        bool fresh = true;  // nothing in the running sum yet
        float z = 0.f;
        // The group of tiles before is emptied when this one's are on their way: its
        // products are done by then, and nothing waits.
        int pending = -1, slot = 0;  // that group, and the state it completes
        bool whole = false;
        long long state = 0;
        auto drain = [&]() {
            const int g = pending;
            wait_bar(&sm.acc_full[g & 1], (g >> 1) & 1, cx);
            tc_fence_after();
            uint32_t v[Sum::kCols];
            float zg = 0.f;
            Sum::get(me, (g & 1) * 160, v, zg);
            tc_fence_before();
            arrive_warp(&sm.acc_empty[g & 1]);
            const uint32_t total = me.lane_base + kTotal + me.part * Sum::kCols;
            if (!fresh) {
#pragma unroll
                for (int h = 0; h < Sum::kCols; h += 16) {
                    uint32_t u[16];
                    tmem_get(total + h, u);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[h + e] = __float_as_uint(u2f(v[h + e]) + u2f(u[e]));
                }
                zg += z;
            }
            fresh = whole;
            z = zg;
            if (whole) {
                Sum::write(p, me, state, slot, v, z);
            } else {
                tmem_put(total, v);
                tmem_wait_st();
            }
        };
        for (int j = 0; j < steps; ++j, w.next()) {
            const int st = j % L::STAGES, len = w.len - w.tile * L::TOK;
            if ((j & 1) == me.group) {
                uint8_t *kt = smem + st * L::STAGE, *vt = kt + L::TILE;
                uint8_t *lt = smem + L::OFF_LOW + j % L::LOWS * L::TILE;
                wait_bar(&sm.full[st], (j / L::STAGES) & 1, cx);
                uint4 u[kChunks];
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
                    u[i] = *reinterpret_cast<const uint4 *>(
                        kt + tile_at(L::TOK, row, (part * kChunks + i) * 8));
                wait_bar(&sm.low_empty[j % L::LOWS], ((j / L::LOWS) & 1) ^ 1, cx);
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    const int col = (part * kChunks + i) * 8;
                    const uint32_t at = tile_at(L::TOK, row, col);
                    float e[8];
                    open8(u[i], e);
                    phi8(e, p.phi);
                    uint4 high = shut8(e), low = low8(e, high);
                    if (row >= len || col >= p.d) high = low = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(kt + at) = high;
                    *reinterpret_cast<uint4 *>(lt + at) = low;
                    if (row >= len)
                        *reinterpret_cast<uint4 *>(vt + at) = make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();
                arrive_warp(&sm.ready[st]);
            }
            if (++in == L::GROUP || w.last() || j == steps - 1) {
                if (pending >= 0) drain();
                const bool began = first > 0, ends = w.last();
                pending = g;
                whole = ends || j == steps - 1;
                slot = began ? 0 : ends ? -1 : 1;
                state = (long long)w.b * p.Hk + w.seg;
                if (whole) {
                    if (began && me.et == 0) {
                        const long long s0 = x.x0 + j - w.tile;
                        p.info[blockIdx.x] =
                            make_int4((int)state, x.of(s0), x.of(s0 + w.tiles - 1), 0);
                    }
                    first = 0;
                }
                ++g;
                in = 0;
            }
        }
        if (pending >= 0) drain();
    }
    end(tmem);
}

// Adds the parts of states that lie in several blocks: blockIdx.y + 1 is the first block
// that continues a state.
__global__ void __launch_bounds__(256) join_parts_kernel(const Params p) {
    grid_dep_launch();
    grid_dep_wait();
    const int i = blockIdx.y + 1;
    const int4 info = p.info[i];
    if (info.x < 0 || info.y != i - 1) return;
    const long long dd = (long long)p.d * p.d, all = dd + p.d;
    const long long e = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= all) return;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int q = info.y; q <= info.z; ++q) {
        const float4 u = __ldcg(
            reinterpret_cast<const float4 *>(p.part + (2 * (long long)q + (q == info.y)) * all + e));
        t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
    }
    float *to = e < dd ? p.So + info.x * dd + e : p.zo + (long long)info.x * p.d + (e - dd);
    *reinterpret_cast<float4 *>(to) = t;
}

// ------------------------------------------------------------------ read
//
// 128 tokens x d of queries stay in their place as phi(q), then as the outputs; two groups
// of computing warps take tiles in turn, so that one works while the other waits.
// 4 x 32 x 4096 x 128 (134 MB in, 134 MB out): 50 us, 5.4 TB/s.

template <int DK>
struct ReadLayout {
    static constexpr int KB = DK / 64, TILE = KB * 16384, STAGES = DK == 128 ? 4 : 8;
    static constexpr int SATOM = DK * 128;  // rows are features a
    // S and behind it the columns of z, one operand of DK + 16 columns
    static constexpr int OFF_S = STAGES * TILE, OFF_Z = OFF_S + KB * SATOM;
    static constexpr int OFF_SMALL = OFF_Z + SATOM;
};
struct ReadSmall {
    uint64_t full[8], empty[8], ready[8], out[8], s_ready, o_full[2], o_empty[2], fin;
    long long plan[kThreads / 32 + 2];
    uint32_t tmem;
    int abort;
};

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
read_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap to,
            const Params p) {
    using L = ReadLayout<DK>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                ~uintptr_t(1023));
    ReadSmall &sm = *reinterpret_cast<ReadSmall *>(smem + L::OFF_SMALL);
    clear(smem + L::OFF_Z, L::SATOM);
    const int tiles = (p.L + 127) / 128;  // of a head of queries
    const uint32_t tmem = begin(&sm.tmem, [&] {
        sm.abort = 0;
        for (int i = 0; i < L::STAGES; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
            mbar_init(&sm.ready[i], kWarpsG);
            mbar_init(&sm.out[i], kWarpsG);
        }
        mbar_init(&sm.s_ready, kWarpsC);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.o_empty[i], kWarpsG);
        }
        mbar_init(&sm.fin, 1);
    });
    const Ctx cx{&sm.abort, p.status, p.timeout};
    auto count = [&](int) { return p.G * tiles; };
    const Piece x = even_piece(p.B, p.Hk, 1, p.G * tiles);
    const int steps = (int)(x.x1 - x.x0);
    auto w = walk(count, p, x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_first();
            int j = 0;
            for (; j < steps; ++j, w.next()) {
                const int st = j % L::STAGES, g = w.tile / tiles;
                if (!may_fetch(p, &sm.empty[st], ((j / L::STAGES) & 1) ^ 1, j, cx)) break;
                mbar_arrive_expect_tx(&sm.full[st], L::TILE);
                for (int a = 0; a < L::KB; ++a)
                    load_tile(smem + st * L::TILE + a * 16384, &tq, &sm.full[st], 64 * a,
                              (w.tile - g * tiles) * 128, w.seg * p.G + g, w.b, pol);
            }
            for (int i = max(0, j - L::STAGES); i < j; ++i)
                settle_wait(&sm.full[i % L::STAGES], (i / L::STAGES) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t id = idesc_bf16(128, DK + 16, 0, 1);
            const uint32_t sb = smem_u32(smem + L::OFF_S);
            int states = 0;
            for (int j = 0; j < steps; ++j, w.next()) {
                const int st = j % L::STAGES;
                if (j == 0 || w.tile == 0) wait_bar_spin(&sm.s_ready, states++ & 1, cx);
                wait_bar_spin(&sm.ready[st], (j / L::STAGES) & 1, cx);
                wait_bar_spin(&sm.o_empty[j & 1], ((j >> 1) & 1) ^ 1, cx);
                tc_fence_after();
                const uint32_t qb = smem_u32(smem + st * L::TILE), o = tmem + (j & 1) * 160;
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks)
                    mma_ss(o, sdesc_sw128(qb + kmajor_off(ks, 16384), 16, 1024),
                           sdesc_sw128(sb + ks * 2048, L::SATOM, 1024), id, ks > 0);
                mma_commit(&sm.o_full[j & 1]);
            }
            mma_commit(&sm.fin);
            settle_wait(&sm.fin, 0);
        }
    } else if (warp < 2 + kWarpsC) {
        const Mine me(tmem);
        constexpr int kChunks = DK / 16;
        const int row = me.et & 127, half = me.part & 1;  // of the tile that the group has
        for (int j = 0; j < steps; ++j, w.next()) {
            const int st = j % L::STAGES;
            if (j == 0 || w.tile == 0) {
                // another state: the products with the one before are done, all their
                // outputs having been taken
                Loaded<DK> S;
                const long long state = (long long)w.b * p.Hk + w.seg;
                S.load(p.S + state * p.d * p.d, p.d, me.et);
                const float z = me.et < p.d ? __ldcg(p.z + state * p.d + me.et) : 0.f;
                sync_compute();
#pragma unroll
                for (int i = 0; i < S.kN; ++i) {
                    float e[8];
                    S.get(i, e);
                    *reinterpret_cast<uint4 *>(smem + L::OFF_S +
                                               tile_at(DK, S.row(me.et, i), S.col(me.et, i))) =
                        shut8(e);
                }
                if (me.et < DK)
                    *reinterpret_cast<uint32_t *>(smem + L::OFF_Z + sw128_offset(me.et, 0)) =
                        split(z);
                fence_async_shared();
                arrive_warp(&sm.s_ready);
            }
            if ((j & 1) != me.group) continue;
            wait_bar(&sm.full[st], (j / L::STAGES) & 1, cx);
            uint8_t *tile = smem + st * L::TILE;
            uint4 u[kChunks];
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                u[i] = *reinterpret_cast<const uint4 *>(
                    tile + tile_at(128, row, (half * kChunks + i) * 8));
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int col = (half * kChunks + i) * 8;
                float e[8];
                open8(u[i], e);
                phi8(e, p.phi);
                *reinterpret_cast<uint4 *>(tile + tile_at(128, row, col)) =
                    col < p.d ? shut8(e) : make_uint4(0, 0, 0, 0);
            }
            fence_async_shared();
            arrive_warp(&sm.ready[st]);

            wait_bar(&sm.o_full[j & 1], (j >> 1) & 1, cx);
            tc_fence_after();
            const uint32_t o = me.lane_base + (j & 1) * 160;
            float inv = 1.f;
            bool none = false;
            if (p.norm) {
                uint32_t d0 = tmem_ld1(o + DK), d1 = tmem_ld1(o + DK + 1);
                tmem_wait_ld();
                reg_fence(d0);
                reg_fence(d1);
                const float den = u2f(d0) + u2f(d1);
                none = den == 0.f;
                inv = none ? 0.f : 1.f / den;
            }
#pragma unroll
            for (int h = 0; h < DK / 64; ++h) {
                uint32_t v[32];
                tmem_get(o + half * (DK / 2) + 32 * h, v);
                if (h == DK / 64 - 1) {
                    tc_fence_before();
                    arrive_warp(&sm.o_empty[j & 1]);
                }
                if (none)
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float e[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) e[q] = u2f(v[8 * i + q]) * inv;
                    *reinterpret_cast<uint4 *>(
                        tile + tile_at(128, me.row, half * (DK / 2) + 32 * h + 8 * i)) = shut8(e);
                }
            }
            fence_async_shared();
            arrive_warp(&sm.out[st]);
        }
    } else if (lane == 0) {
        for (int j = 0; j < steps; ++j, w.next()) {
            const int st = j % L::STAGES, g = w.tile / tiles;
            if (!wait_bar(&sm.out[st], (j / L::STAGES) & 1, cx)) break;
            for (int a = 0; a < L::KB; ++a)
                if (64 * a < p.d)
                    store_tile(&to, smem + st * L::TILE + a * 16384, 64 * a,
                               (w.tile - g * tiles) * 128, w.seg * p.G + g, w.b);
            tma_store_commit();
            tma_store_wait_read<0>();
            mbar_arrive(&sm.empty[st]);
        }
        tma_store_wait_all<0>();
    }
    end(tmem);
}

// ------------------------------------------------------------------ qgrad
//
// Two products depend on one another for each tile (psi needs the first's t), and the
// second's sums stay in TMEM over up to 16 tiles of a state: then they are added to those
// before in memory, by reductions that nothing waits for.  4 x 8 x 4096 x 128 (101 MB in and
// out): 42 us, 2.4 TB/s: 7 tiles per block, each at the latency of fetch, product, psi,
// product and store.  Two groups of computing warps 48 us (a state's sums then meet at its end);
// dq straight from registers 51 us.

template <int DK>
struct QLayout {
    static constexpr int KB = DK / 64, TILE = KB * 16384, STAGE = 2 * TILE;
    static constexpr int STAGES = DK == 128 ? 2 : 4;
    static constexpr int SROWS = DK + 16, SATOM = SROWS * 128;  // rows of S', then m
    // Tiles of a chain of sums.  2048 tokens are 128 products, of which the cut takes 2^-16 at
    // most, as much as dS loses in two bf16 numbers; over a million tokens without an end dk
    // was off by 7 % where values have a mean of 64 deviations.  20 x (32 on 8) x 16384 to
    // 2048 x 64 backward: 949 us without an end, 975 us with 16; 4 take 84 us more.
    static constexpr int GROUP = 16;
    static constexpr int OFF_T = STAGES * STAGE, OFF_S = OFF_T + 16384;
    static constexpr int OFF_OUT = (OFF_S + KB * SATOM + 1023) / 1024 * 1024;
    static constexpr int OFF_SMALL = OFF_OUT + TILE;
};
struct QSmall {
    uint64_t full[4], y_full[4], empty[4], psi[4], s_ready, g_full[2], g_empty[2], t_free, ds_full, ds_empty;
    uint64_t out_full, out_empty, fin;
    long long plan[kThreads / 32 + 2];
    float z[128], m[128];
    union {
        float2 red[2][kC];
        float sum[kWarpsC][128];
    };
    uint32_t tmem;
    int abort;
};

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
qgrad_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdy,
             const __grid_constant__ CUtensorMap tdq, const Params p) {
    using L = QLayout<DK>;
    constexpr uint32_t kTmG = 0, kTmStep = 144, kDs = 288;  // TMEM columns
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                ~uintptr_t(1023));
    QSmall &sm = *reinterpret_cast<QSmall *>(smem + L::OFF_SMALL);
    clear(smem + L::OFF_T, 16384);
    clear(smem + L::OFF_S, L::KB * L::SATOM);
    const int tiles = (p.L + 127) / 128;
    const uint32_t tmem = begin(&sm.tmem, [&] {
        sm.abort = 0;
        for (int i = 0; i < L::STAGES; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.y_full[i], 1);
            mbar_init(&sm.empty[i], 1);
            mbar_init(&sm.psi[i], kWarpsC);
        }
        mbar_init(&sm.s_ready, kWarpsC);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.g_full[i], 1);
            mbar_init(&sm.g_empty[i], kWarpsC);
        }
        mbar_init(&sm.t_free, 1);
        mbar_init(&sm.ds_full, 1);
        mbar_init(&sm.ds_empty, kWarpsC);
        mbar_init(&sm.out_full, kWarpsC);
        mbar_init(&sm.out_empty, 1);
        mbar_init(&sm.fin, 1);
    });
    const Ctx cx{&sm.abort, p.status, p.timeout};
    auto count = [&](int) { return p.G * tiles; };
    const Piece x = even_piece(p.B, p.Hk, 2, p.G * tiles);
    const int steps = (int)(x.x1 - x.x0);
    if (threadIdx.x == 0) p.info[blockIdx.x] = make_int4(-1, 0, 0, 0);
    auto w = walk(count, p, x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_first();
            int j = 0;
            for (; j < steps; ++j, w.next()) {
                const int st = j % L::STAGES, g = w.tile / tiles;
                if (!may_fetch(p, &sm.empty[st], ((j / L::STAGES) & 1) ^ 1, j, cx)) break;
                // the first product needs dY alone: it comes first and is waited for apart
                mbar_arrive_expect_tx(&sm.y_full[st], L::TILE);
                mbar_arrive_expect_tx(&sm.full[st], L::TILE);
                uint8_t *at = smem + st * L::STAGE;
                const int tok = (w.tile - g * tiles) * 128, h = w.seg * p.G + g;
                for (int a = 0; a < L::KB; ++a)
                    load_tile(at + L::TILE + a * 16384, &tdy, &sm.y_full[st], 64 * a, tok, h, w.b,
                              pol);
                for (int a = 0; a < L::KB; ++a)
                    load_tile(at + a * 16384, &tq, &sm.full[st], 64 * a, tok, h, w.b, pol);
            }
            for (int i = max(0, j - L::STAGES); i < j; ++i) {
                settle_wait(&sm.full[i % L::STAGES], (i / L::STAGES) & 1);
                settle_wait(&sm.y_full[i % L::STAGES], (i / L::STAGES) & 1);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idG = idesc_bf16(128, DK + 16, 0, 0);
            constexpr uint32_t id0 = idesc_bf16(128, 80, 1, 1), id1 = idesc_bf16(128, 64, 1, 1);
            constexpr uint32_t lboA = DK == 128 ? 16384 : 0;
            const uint32_t sb = smem_u32(smem + L::OFF_S), tb = smem_u32(smem + L::OFF_T);
            // G of tile i and the sums of tile j <= i, whichever has its operands: a tile
            // that is still under way holds back no sums, which free a place for the next
            auto v = w;
            int i = 0, j = 0, states = 0, ended = 0, in = 0;
            long long deadline = 0;
            for (int polls = 0; j < steps;) {
                if (j < i) {
                    const int st = j % L::STAGES;
                    const bool first = in == 0;
                    const bool last = v.last() || j == steps - 1 || in == L::GROUP - 1;
                    if (mbar_test_wait(&sm.psi[st], (j / L::STAGES) & 1) &&
                        (!first || mbar_test_wait(&sm.ds_empty, (ended & 1) ^ 1))) {
                        tc_fence_after();
                        const uint32_t qb = smem_u32(smem + st * L::STAGE), yb = qb + L::TILE;
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint64_t a = sdesc_sw128(qb + ks * 2048, lboA, 1024);
                            const uint32_t more = !first || ks > 0;
                            mma_ss(tmem + kDs, a, sdesc_sw128(yb + ks * 2048, tb - yb, 1024), id0,
                                   more);
                            if (DK == 128)
                                mma_ss(tmem + kDs + 80, a,
                                       sdesc_sw128(yb + 16384 + ks * 2048, 0, 1024), id1, more);
                        }
                        mma_commit(&sm.empty[st]);
                        mma_commit(&sm.t_free);
                        ++in;
                        if (last) {
                            mma_commit(&sm.ds_full);
                            ++ended;
                            in = 0;
                        }
                        ++j;
                        v.next();
                        polls = 0;
                        continue;
                    }
                }
                if (i < steps) {
                    const int st = i % L::STAGES;
                    const bool first = i == 0 || w.tile == 0;
                    if (mbar_test_wait(&sm.y_full[st], (i / L::STAGES) & 1) &&
                        mbar_test_wait(&sm.g_empty[i & 1], ((i >> 1) & 1) ^ 1) &&
                        (!first || mbar_test_wait(&sm.s_ready, states & 1))) {
                        tc_fence_after();
                        const uint32_t yb = smem_u32(smem + st * L::STAGE + L::TILE);
#pragma unroll
                        for (int ks = 0; ks < DK / 16; ++ks)
                            mma_ss(tmem + kTmG + (i & 1) * kTmStep,
                                   sdesc_sw128(yb + kmajor_off(ks, 16384), 16, 1024),
                                   sdesc_sw128(sb + kmajor_off(ks, L::SATOM), 16, 1024), idG,
                                   ks > 0);
                        mma_commit(&sm.g_full[i & 1]);
                        states += first;
                        ++i;
                        w.next();
                        polls = 0;
                        continue;
                    }
                }
                if ((++polls & 63) == 0) {
                    if (*cx.abort) break;
                    const long long now = clock64();
                    if (polls == 64) deadline = now + cx.timeout;
                    if (now > deadline) {
                        raise_timeout(cx, smem_u32(&sm.psi[0]));
                        break;
                    }
                }
            }
            mma_commit(&sm.fin);
            settle_wait(&sm.fin, 0);
        }
    } else if (warp < 2 + kWarpsC) {
        const Mine me(tmem);
        constexpr int kCols = DK / kParts;
        const int f0 = me.part * kCols;  // this thread's features of its row
        int first_tile = w.tile, drained = 0;
        // the chain of sums that has ended, if >= 0: its state, where it goes to, and whether
        // one before it is there
        int old_state = -1, old_slot = 0;
        bool old_more = false;
        auto drain = [&]() {
            wait_bar(&sm.ds_full, drained & 1, cx);
            ++drained;
            tc_fence_after();
            using Sum = Sums<DK, 64, 2>;
            uint32_t v[Sum::kCols];
            float z = 0.f;
            Sum::get(me, kDs, v, z);
            tc_fence_before();
            arrive_warp(&sm.ds_empty);
            Sum::write(p, me, old_state, old_slot, v, z, old_more);
            old_state = -1;
        };
        for (int j = 0; j < steps; ++j, w.next()) {
            const int st = j % L::STAGES;
            const long long state = (long long)w.b * p.Hk + w.seg;
            if (j == 0 || w.tile == 0) {
                Loaded<DK> S;
                // (without the normaliser z is no part of the formulas, whatever it is)
                const float z_mine =
                    p.norm && me.et < p.d ? __ldcg(p.z + state * p.d + me.et) : 0.f;
                S.load(p.S + state * p.d * p.d, p.d, me.et);
                sync_compute();  // all are through with the state before
                if (me.et < 128) sm.z[me.et] = z_mine;
                sync_compute();
                // m = S^T z / z.z; the threads of a column chunk are DK / 8 apart
                float zz = 0.f, mine[8] = {};
                for (int a = lane; a < DK; a += 32) zz = fmaf(sm.z[a], sm.z[a], zz);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) zz += __shfl_xor_sync(~0u, zz, o);
#pragma unroll
                for (int i = 0; i < S.kN; ++i) {
                    float e[8];
                    S.get(i, e);
                    const float za = sm.z[S.row(me.et, i)];
#pragma unroll
                    for (int q = 0; q < 8; ++q) mine[q] = fmaf(e[q], za, mine[q]);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
#pragma unroll
                    for (int o = DK / 8; o < 32; o <<= 1)
                        mine[q] += __shfl_xor_sync(~0u, mine[q], o);
                if (lane < DK / 8)
#pragma unroll
                    for (int q = 0; q < 8; ++q) sm.sum[me.et >> 5][lane * 8 + q] = mine[q];
                sync_compute();
                if (me.et < DK) {
                    float t = 0.f;
#pragma unroll
                    for (int q = 0; q < kWarpsC; ++q) t += sm.sum[q][me.et];
                    sm.m[me.et] = zz > 0.f && p.norm ? t / zz : 0.f;
                }
                sync_compute();
#pragma unroll
                for (int i = 0; i < S.kN; ++i) {
                    float e[8];
                    S.get(i, e);
                    const int a = S.row(me.et, i), c = S.col(me.et, i);
                    const float z = sm.z[a];
#pragma unroll
                    for (int q = 0; q < 8; ++q) e[q] = fmaf(-z, sm.m[c + q], e[q]);
                    *reinterpret_cast<uint4 *>(smem + L::OFF_S + tile_at(L::SROWS, a, c)) = shut8(e);
                }
                if (me.et < DK) {  // row DK: m, row DK + 1: what it loses
                    const float m = me.et < p.d ? sm.m[me.et] : 0.f;
                    const uint32_t both = split(m);
                    uint8_t *at = smem + L::OFF_S + (me.et >> 6) * L::SATOM;
                    *reinterpret_cast<uint16_t *>(at + sw128_offset(DK, me.et & 63)) =
                        (uint16_t)both;
                    *reinterpret_cast<uint16_t *>(at + sw128_offset(DK + 1, me.et & 63)) =
                        (uint16_t)(both >> 16);
                }
                fence_async_shared();
                arrive_warp(&sm.s_ready);
                first_tile = w.tile;
            }
            wait_bar(&sm.full[st], (j / L::STAGES) & 1, cx);
            uint8_t *qt = smem + st * L::STAGE;
            // phi(q), its product with z and, behind the products' end, with G
            float f[kCols], den = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < kCols; i += 8) {
                float e[8];
                open8(*reinterpret_cast<const uint4 *>(qt + tile_at(128, me.row, f0 + i)), e);
                phi8(e, p.phi);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    f[i + q] = f0 + i < p.d ? e[q] : 0.f;
                    den = fmaf(f[i + q], sm.z[f0 + i + q], den);
                }
            }
            if (old_state >= 0) drain();  // of the tiles before: phi has given it time
            wait_bar(&sm.g_full[j & 1], (j >> 1) & 1, cx);
            tc_fence_after();
            const uint32_t gb = me.lane_base + kTmG + (j & 1) * kTmStep;
            uint32_t v[kCols];
            tmem_get(gb + f0, v);
#pragma unroll
            for (int e = 0; e < kCols; ++e) dot = fmaf(f[e], u2f(v[e]), dot);
            uint32_t m0 = tmem_ld1(gb + DK), m1 = tmem_ld1(gb + DK + 1);
            tmem_wait_ld();
            reg_fence(m0);
            reg_fence(m1);
            tc_fence_before();
            arrive_warp(&sm.g_empty[j & 1]);
            sm.red[j & 1][me.part * 128 + me.row] = make_float2(den, dot);
            // the staging tile and t's column are free again
            wait_bar(&sm.out_empty, (j & 1) ^ 1, cx);
            wait_bar(&sm.t_free, (j & 1) ^ 1, cx);
            sync_compute();
            den = dot = 0.f;
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
                const float2 r = sm.red[j & 1][128 * q + me.row];
                den += r.x;
                dot += r.y;
            }
            float r = 1.f, t = 0.f, t_all = 0.f;
            if (p.norm) {
                r = 1.f / den;
                t = dot * r;
                t_all = t + u2f(m0) + u2f(m1);
            }
            uint8_t *ot = smem + L::OFF_OUT;
#pragma unroll
            for (int i = 0; i < kCols; i += 8) {
                float g[8], s[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    g[q] = r * fmaf(-t, sm.z[f0 + i + q], u2f(v[i + q])) *
                           slope_of_phi(f[i + q], p.phi);
                    s[q] = r * f[i + q];
                }
                const uint32_t at = tile_at(128, me.row, f0 + i);
                *reinterpret_cast<uint4 *>(ot + at) = shut8(g);
                *reinterpret_cast<uint4 *>(qt + at) = shut8(s);
            }
            if (p.norm && den == 0.f) {
                // the row's gradient is 0 and it adds nothing, whatever S and its dY are (G
                // has been formed of that); rare, and apart from the way of the others
                t_all = 0.f;
                for (int i = 0; i < kCols; i += 8) {
                    const uint32_t at = tile_at(128, me.row, f0 + i);
                    *reinterpret_cast<uint4 *>(ot + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(qt + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(qt + L::TILE + at) = make_uint4(0, 0, 0, 0);
                }
            }
            if (me.part == 0)
                *reinterpret_cast<uint32_t *>(smem + L::OFF_T + sw128_offset(me.row, 0)) =
                    split(t_all);
            fence_async_shared();
            arrive_warp(&sm.psi[st]);
            if (lane == 0) mbar_arrive(&sm.out_full);
            const bool whole = w.last() || j == steps - 1;
            const int at = w.tile - first_tile;
            if (whole || at % L::GROUP == L::GROUP - 1) {
                const bool began = first_tile > 0, ends = w.tiles - w.tile <= steps - j;
                old_state = (int)state;
                old_slot = began ? 0 : ends ? -1 : 1;
                old_more = at >= L::GROUP;
                if (whole && began && me.et == 0) {
                    const long long s0 = x.x0 + j - w.tile;
                    p.info[blockIdx.x] =
                        make_int4((int)state, x.of(s0), x.of(s0 + w.tiles - 1), 0);
                }
            }
        }
        if (old_state >= 0) drain();
    } else if (lane == 0) {
        for (int j = 0; j < steps; ++j, w.next()) {
            const int g = w.tile / tiles;
            if (!wait_bar(&sm.out_full, j & 1, cx)) break;
            for (int a = 0; a < L::KB; ++a)
                if (64 * a < p.d)
                    store_tile(&tdq, smem + L::OFF_OUT + a * 16384, 64 * a,
                               (w.tile - g * tiles) * 128, w.seg * p.G + g, w.b);
            tma_store_commit();
            tma_store_wait_read<0>();
            mbar_arrive(&sm.out_empty);
        }
        tma_store_wait_all<0>();
    }
    end(tmem);
}

// ------------------------------------------------------------------ kgrad
//
// dphi(K) goes into K's place and dV into V's, after the products that read them; two
// groups of computing warps take tiles in turn.  4 x 8 x 16384 x 128 (ragged; 198 MB in,
// 268 MB out with the padding's zeros): 94 us, 5.0 TB/s.  Both gradients straight from
// registers 144 us; staged in halves with phi in place 136 us.

template <int DK>
struct KLayout {
    static constexpr int KB = DK / 64, TILE = KB * 16384, STAGE = 2 * TILE;
    static constexpr int STAGES = DK == 128 ? 2 : 4;
    static constexpr int SATOM = DK * 128, SBLK = KB * SATOM;
    static constexpr int OFF_PHI = STAGES * STAGE, OFF_S = OFF_PHI + TILE;
    static constexpr int OFF_SMALL = OFF_S + 2 * SBLK;
    static_assert(2 * SBLK >= 16384, "a tile of zeros fits");
};
struct KSmall {
    uint64_t full[4], v_full[4], empty[4], ready[4], out[4], s_ready, phi_empty, dk_full[2], dv_full[2],
        d_empty[2], fin;
    long long plan[kThreads / 32 + 2];
    float dz[128];
    uint32_t tmem;
    int abort;
};

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
kgrad_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
             const __grid_constant__ CUtensorMap tdk, const __grid_constant__ CUtensorMap tdv,
             const Params p) {
    using L = KLayout<DK>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                ~uintptr_t(1023));
    KSmall &sm = *reinterpret_cast<KSmall *>(smem + L::OFF_SMALL);
    const uint32_t tmem = begin(&sm.tmem, [&] {
        sm.abort = 0;
        for (int i = 0; i < L::STAGES; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.empty[i], 1);
            mbar_init(&sm.ready[i], kWarpsG);
            mbar_init(&sm.out[i], kWarpsG);
        }
        mbar_init(&sm.s_ready, kWarpsC);
        mbar_init(&sm.phi_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.dk_full[i], 1);
            mbar_init(&sm.dv_full[i], 1);
            mbar_init(&sm.d_empty[i], kWarpsG);
        }
        mbar_init(&sm.fin, 1);
    });
    const Ctx cx{&sm.abort, p.status, p.timeout};
    auto count = [](int len) { return (len + 127) / 128; };
    const Piece x = find_piece<kThreads>(
        p.B, p.Hk, 1, [&](int b) { return count(tokens_of(p, b)); }, sm.plan);
    const int steps = (int)(x.x1 - x.x0);
    auto w = walk(count, p, x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_first();
            int j = 0;
            for (; j < steps; ++j, w.next()) {
                const int st = j % L::STAGES;
                if (!may_fetch(p, &sm.empty[st], ((j / L::STAGES) & 1) ^ 1, j, cx)) break;
                // phi needs the keys alone: they come first and are waited for apart
                mbar_arrive_expect_tx(&sm.full[st], L::TILE);
                mbar_arrive_expect_tx(&sm.v_full[st], L::TILE);
                uint8_t *at = smem + st * L::STAGE;
                for (int a = 0; a < L::KB; ++a)
                    load_tile(at + a * 16384, &tk, &sm.full[st], 64 * a, w.tile * 128, w.seg, w.b,
                              pol);
                for (int a = 0; a < L::KB; ++a)
                    load_tile(at + L::TILE + a * 16384, &tv, &sm.v_full[st], 64 * a, w.tile * 128,
                              w.seg, w.b, pol);
            }
            for (int i = max(0, j - L::STAGES); i < j; ++i) {
                settle_wait(&sm.full[i % L::STAGES], (i / L::STAGES) & 1);
                settle_wait(&sm.v_full[i % L::STAGES], (i / L::STAGES) & 1);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idK = idesc_bf16(128, DK, 0, 0), idV = idesc_bf16(128, DK, 0, 1);
            const uint32_t hi = smem_u32(smem + L::OFF_S), lo = hi + L::SBLK;
            // dphi(K) of tile i needs V alone, dV of tile j <= i needs phi(K): whichever has
            // its operands
            int i = 0, j = 0, states = 0;
            long long deadline = 0;
            for (int polls = 0; j < steps;) {
                if (j < i && mbar_test_wait(&sm.ready[j % L::STAGES], (j / L::STAGES) & 1)) {
                    tc_fence_after();
                    const uint32_t dv = tmem + (j & 1) * 2 * DK + DK;
                    const uint32_t fb = smem_u32(smem + L::OFF_PHI);
#pragma unroll
                    for (int ks = 0; ks < DK / 16; ++ks)
                        mma_ss(dv, sdesc_sw128(fb + kmajor_off(ks, 16384), 16, 1024),
                               sdesc_sw128(hi + ks * 2048, L::SATOM, 1024), idV, ks > 0);
                    mma_commit(&sm.phi_empty);
                    mma_commit(&sm.dv_full[j & 1]);
                    ++j;
                    polls = 0;
                    continue;
                }
                if (i < steps) {
                    const int st = i % L::STAGES;
                    const bool first = i == 0 || w.tile == 0;
                    if (mbar_test_wait(&sm.v_full[st], (i / L::STAGES) & 1) &&
                        mbar_test_wait(&sm.d_empty[i & 1], ((i >> 1) & 1) ^ 1) &&
                        (!first || mbar_test_wait(&sm.s_ready, states & 1))) {
                        tc_fence_after();
                        const uint32_t vb = smem_u32(smem + st * L::STAGE + L::TILE);
                        const uint32_t dk = tmem + (i & 1) * 2 * DK;
#pragma unroll
                        for (int ks = 0; ks < DK / 16; ++ks) {
                            const uint64_t a = sdesc_sw128(vb + kmajor_off(ks, 16384), 16, 1024);
                            mma_ss(dk, a, sdesc_sw128(hi + kmajor_off(ks, L::SATOM), 16, 1024),
                                   idK, ks > 0);
                            mma_ss(dk, a, sdesc_sw128(lo + kmajor_off(ks, L::SATOM), 16, 1024),
                                   idK, 1);
                        }
                        mma_commit(&sm.dk_full[i & 1]);
                        states += first;
                        ++i;
                        w.next();
                        polls = 0;
                        continue;
                    }
                }
                if ((++polls & 63) == 0) {
                    if (*cx.abort) break;
                    const long long now = clock64();
                    if (polls == 64) deadline = now + cx.timeout;
                    if (now > deadline) {
                        raise_timeout(cx, smem_u32(&sm.ready[0]));
                        break;
                    }
                }
            }
            mma_commit(&sm.fin);
            settle_wait(&sm.fin, 0);
        }
    } else if (warp < 2 + kWarpsC) {
        const Mine me(tmem);
        constexpr int kChunks = DK / 16;
        const int row = me.row, half = me.part & 1, f0 = half * (DK / 2);
        for (int j = 0; j < steps; ++j, w.next()) {
            const int st = j % L::STAGES, len = w.len - w.tile * 128;
            if (j == 0 || w.tile == 0) {
                Loaded<DK> S;
                const long long state = (long long)w.b * p.Hk + w.seg;
                S.load(p.S + state * p.d * p.d, p.d, me.et);
                const float dz = me.et < p.d ? __ldcg(p.z + state * p.d + me.et) : 0.f;
                sync_compute();  // all are through with the state before
#pragma unroll
                for (int i = 0; i < S.kN; ++i) {
                    float e[8];
                    S.get(i, e);
                    uint8_t *at =
                        smem + L::OFF_S + tile_at(DK, S.row(me.et, i), S.col(me.et, i));
                    const uint4 high = shut8(e);
                    *reinterpret_cast<uint4 *>(at) = high;
                    *reinterpret_cast<uint4 *>(at + L::SBLK) = low8(e, high);
                }
                if (me.et < 128) sm.dz[me.et] = dz;
                fence_async_shared();
                sync_compute();
                arrive_warp(&sm.s_ready);
            }
            if ((j & 1) != me.group) continue;
            wait_bar(&sm.full[st], (j / L::STAGES) & 1, cx);
            uint8_t *kt = smem + st * L::STAGE, *vt = kt + L::TILE;
            uint4 u[kChunks];
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                u[i] = *reinterpret_cast<const uint4 *>(
                    kt + tile_at(128, row, (half * kChunks + i) * 8));
            const bool whole_tile = len >= 128 && p.d == DK;
            wait_bar(&sm.phi_empty, (j & 1) ^ 1, cx);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int col = (half * kChunks + i) * 8;
                const uint32_t at = tile_at(128, row, col);
                float e[8];
                open8(u[i], e);
                phi8(e, p.phi);
                uint4 f = shut8(e);
                if (!whole_tile && (row >= len || col >= p.d)) f = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(smem + L::OFF_PHI + at) = f;
            }
            fence_async_shared();
            arrive_warp(&sm.ready[st]);

            // dk over k, by the threads that have read it; dv over V, which is no operand any
            // more.  What lies behind the length in V stays in its own rows.
            wait_bar(&sm.dk_full[j & 1], (j >> 1) & 1, cx);
            tc_fence_after();
            const uint32_t dk = me.lane_base + (j & 1) * 2 * DK + f0;
#pragma unroll
            for (int h = 0; h < DK / 64; ++h) {
                uint32_t v[32];
                uint4 u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    u[i] = *reinterpret_cast<const uint4 *>(
                        kt + tile_at(128, row, f0 + 32 * h + 8 * i));
                tmem_get(dk + 32 * h, v);
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    float x[8];
                    open8(u[i / 8], x);
#pragma unroll
                    for (int q = 0; q < 8; q += 2) {
                        const float2 dz =
                            *reinterpret_cast<const float2 *>(&sm.dz[f0 + 32 * h + i + q]);
                        float2 g = __fadd2_rn(make_float2(u2f(v[i + q]), u2f(v[i + q + 1])), dz);
                        if (p.phi) g = __fmul2_rn(g, exp_below(make_float2(x[q], x[q + 1])));
                        x[q] = g.x;
                        x[q + 1] = g.y;
                    }
                    *reinterpret_cast<uint4 *>(kt + tile_at(128, row, f0 + 32 * h + i)) =
                        row < len ? shut8(x) : make_uint4(0, 0, 0, 0);
                }
            }
            wait_bar(&sm.dv_full[j & 1], (j >> 1) & 1, cx);
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < DK / 64; ++h) {
                uint32_t v[32];
                tmem_get(dk + DK + 32 * h, v);
                if (h == DK / 64 - 1) {
                    tc_fence_before();
                    arrive_warp(&sm.d_empty[j & 1]);
                }
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    float o[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) o[q] = u2f(v[i + q]);
                    // (0 times dS is not 0 where dS is not finite)
                    *reinterpret_cast<uint4 *>(vt + tile_at(128, row, f0 + 32 * h + i)) =
                        row < len ? shut8(o) : make_uint4(0, 0, 0, 0);
                }
            }
            fence_async_shared();
            arrive_warp(&sm.out[st]);
        }
    } else if (lane == 0) {
        for (int j = 0; j < steps; ++j, w.next()) {
            const int st = j % L::STAGES;
            if (!wait_bar(&sm.out[st], (j / L::STAGES) & 1, cx)) break;
            uint8_t *at = smem + st * L::STAGE;
            for (int a = 0; a < L::KB; ++a)
                if (64 * a < p.d) {
                    store_tile(&tdk, at + a * 16384, 64 * a, w.tile * 128, w.seg, w.b);
                    store_tile(&tdv, at + L::TILE + a * 16384, 64 * a, w.tile * 128, w.seg, w.b);
                }
            tma_store_commit();
            tma_store_wait_read<0>();
            mbar_arrive(&sm.empty[st]);
        }
    }
    // tiles that are padding alone: zeros
    __syncthreads();
    if (p.lengths) {
        const int all = (p.L + 127) / 128;
        auto pads = [&](int len) { return all - (len + 127) / 128; };
        const Piece y = find_piece<kThreads>(
            p.B, p.Hk, 1, [&](int b) { return pads(tokens_of(p, b)); }, sm.plan);
        clear(smem + L::OFF_S, 16384);
        fence_async_shared();
        __syncthreads();
        if (warp == 2 + kWarpsC && lane == 0) {
            auto v = walk(pads, p, y);
            for (long long i = y.x0; i < y.x1; ++i, v.next())
                for (int c = 0; c < p.d; c += 64) {
                    const int tok = (all - v.tiles + v.tile) * 128;
                    store_tile(&tdk, smem + L::OFF_S, c, tok, v.seg, v.b);
                    store_tile(&tdv, smem + L::OFF_S, c, tok, v.seg, v.b);
                }
        }
    }
    if (warp == 2 + kWarpsC && lane == 0) {
        tma_store_commit();
        tma_store_wait_all<0>();
    }
    end(tmem);
}

// ------------------------------------------------------------------ host

// Rows of one tensor for tiles of `rows` tokens and 64 features, 128-byte swizzle; what
// lies outside reads as 0 and is not written.
cudaError_t make_map(CUtensorMap *map, const Rows &r, int B, int H, int L, int d, int rows) {
    cudaError_t err;
    auto enc = tchost::encode_fn(&err);
    if (!enc) return err == cudaSuccess ? cudaErrorNotSupported : err;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)H, (cuuint64_t)B};
    // a dimension of one has no stride to go by
    const long long n = L > 1 ? r.s.n : (d + 7) / 8 * 8;
    const long long h = H > 1 ? r.s.h : n, b = B > 1 ? r.s.b : n;
    const cuuint64_t strides[3] = {(cuuint64_t)n * 2, (cuuint64_t)h * 2, (cuuint64_t)b * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUresult e = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r.x, dims, strides, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

bool rows_fit(const Rows &r, int B, int H, int L) {
    if ((uintptr_t)r.x % 16) return false;
    const long long s[3] = {r.s.b, r.s.h, r.s.n};
    const int n[3] = {B, H, L};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] % 8 || s[i] < 8 || s[i] >= 1LL << 38)) return false;
    return true;
}

// How long a call's kernels wait, and the test hook's hold.
struct Limits {
    long long timeout = 1LL << 32;
    int hold = -1;
    Limits() { tc_debug_take_timeout(&timeout, &hold); }
};

Params params_of(const Shape &sh, int L, const Limits &lim, int *status) {
    Params p{};
    p.B = sh.B;
    p.Hk = sh.Hk;
    p.G = sh.G();
    p.L = L;
    p.d = sh.d;
    p.phi = sh.phi;
    p.norm = sh.norm;
    p.zsign = 1.f;
    p.status = status;
    p.timeout = lim.timeout;
    p.hold = lim.hold;
    return p;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Blocks of a kernel over tiles of `tok` of L tokens: no more than there can be.
int blocks_of(const Shape &sh, long long per_state, int sms) {
    return (int)std::max(1LL, std::min((long long)sms, sh.heads() * per_state));
}

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), int blocks, size_t small, int off_small, bool dependent,
                   cudaStream_t s, A &&...args) {
    const size_t smem = (size_t)off_small + small + 1024;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dependent) {
        e = tchost::launch_dependent(kern, dim3((unsigned)blocks), kThreads, smem, s,
                                     std::forward<A>(args)...);
    } else {
        kern<<<(unsigned)blocks, kThreads, smem, s>>>(std::forward<A>(args)...);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) note_launches(1);
    return e;
}

cudaError_t join(const Params &p, int blocks, cudaStream_t s) {
    if (blocks == 1) return cudaSuccess;
    const int all = p.d * p.d + p.d;
    const cudaError_t e =
        tchost::launch_dependent(join_parts_kernel, dim3((unsigned)(all + 1023) / 1024, (unsigned)blocks - 1),
                                 256, 0, s, p);
    if (e == cudaSuccess) note_launches(1);
    return e;
}

template <int DK>
constexpr bool fits() {
    return StateLayout<DK>::OFF_SMALL + sizeof(StateSmall) + 1024 <= 232448 &&
           ReadLayout<DK>::OFF_SMALL + sizeof(ReadSmall) + 1024 <= 232448 &&
           QLayout<DK>::OFF_SMALL + sizeof(QSmall) + 1024 <= 232448 &&
           KLayout<DK>::OFF_SMALL + sizeof(KSmall) + 1024 <= 232448;
}
static_assert(fits<64>() && fits<128>(), "shared memory");

template <int DK>
cudaError_t state(const Shape &sh, Rows k, Rows v, float *S, float *z, char *ws, int sms,
                  int *status, cudaStream_t s) {
    using L = StateLayout<DK>;
    CUtensorMap tk, tv;
    cudaError_t e = make_map(&tk, k, sh.B, sh.Hk, sh.M, sh.d, L::TOK);
    if (e == cudaSuccess) e = make_map(&tv, v, sh.B, sh.Hk, sh.M, sh.d, L::TOK);
    if (e != cudaSuccess) return e;
    Params p = params_of(sh, sh.M, Limits(), status);
    p.lengths = sh.lengths;
    p.So = S;
    p.zo = z;
    p.info = reinterpret_cast<int4 *>(ws);
    p.part = reinterpret_cast<float *>(ws + up(sizeof(int4) * (size_t)sms));
    const int blocks = blocks_of(sh, (sh.M + L::TOK - 1) / L::TOK, sms);
    e = launch(state_kernel<DK>, blocks, sizeof(StateSmall), L::OFF_SMALL, false, s, tk, tv, p);
    return e == cudaSuccess ? join(p, blocks, s) : e;
}

template <int DK>
cudaError_t read(const Shape &sh, Rows q, Rows out, const float *S, const float *z, bool dependent,
                 int sms, int *status, cudaStream_t s) {
    using L = ReadLayout<DK>;
    CUtensorMap tq, to;
    cudaError_t e = make_map(&tq, q, sh.B, sh.Hq, sh.N, sh.d, 128);
    if (e == cudaSuccess) e = make_map(&to, out, sh.B, sh.Hq, sh.N, sh.d, 128);
    if (e != cudaSuccess) return e;
    Params p = params_of(sh, sh.N, Limits(), status);
    p.S = S;
    p.z = z;
    const int blocks = blocks_of(sh, (long long)sh.G() * ((sh.N + 127) / 128), sms);
    return launch(read_kernel<DK>, blocks, sizeof(ReadSmall), L::OFF_SMALL, dependent, s, tq, to, p);
}

template <int DK>
cudaError_t back(const Shape &sh, Rows dout, Rows q, Rows k, Rows v, const float *S,
                 const float *z, Rows dq, Rows dk, Rows dv, char *ws, int sms, int *status,
                 cudaStream_t s) {
    CUtensorMap m[7];
    const Rows *r[7] = {&q, &dout, &dq, &k, &v, &dk, &dv};
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 7 && e == cudaSuccess; ++i)
        e = i < 3 ? make_map(&m[i], *r[i], sh.B, sh.Hq, sh.N, sh.d, 128)
                  : make_map(&m[i], *r[i], sh.B, sh.Hk, sh.M, sh.d, 128);
    if (e != cudaSuccess) return e;
    const Limits lim;  // of both kernels
    Params p = params_of(sh, sh.N, lim, status);
    float *dS = reinterpret_cast<float *>(ws);
    float *dz = reinterpret_cast<float *>(ws + up(sizeof(float) * (size_t)(sh.heads() * sh.state())));
    char *rest = reinterpret_cast<char *>(dz) + up(sizeof(float) * (size_t)(sh.heads() * sh.d));
    p.S = S;
    p.z = z;
    p.So = dS;
    p.zo = dz;
    p.zsign = -1.f;
    p.info = reinterpret_cast<int4 *>(rest);
    p.part = reinterpret_cast<float *>(rest + up(sizeof(int4) * (size_t)sms));
    const int blocks = blocks_of(sh, (long long)sh.G() * ((sh.N + 127) / 128), sms);
    e = launch(qgrad_kernel<DK>, blocks, sizeof(QSmall), QLayout<DK>::OFF_SMALL, false, s, m[0],
               m[1], m[2], p);
    if (e == cudaSuccess) e = join(p, blocks, s);
    if (e != cudaSuccess) return e;
    Params c = params_of(sh, sh.M, lim, status);
    c.lengths = sh.lengths;
    c.S = dS;
    c.z = dz;
    return launch(kgrad_kernel<DK>, blocks_of(sh, (sh.M + 127) / 128, sms), sizeof(KSmall),
                  KLayout<DK>::OFF_SMALL, true, s, m[3], m[4], m[5], m[6], c);
}

}  // namespace

bool tc_rows(const Shape &sh, const Rows *q_side, int nq, const Rows *k_side, int nk,
             const float *S, const float *z) {
    if (sh.d > 128 || sh.d % 8 || (uintptr_t)S % 16 || (uintptr_t)z % 16) return false;
    for (int i = 0; i < nq; ++i)
        if (!rows_fit(q_side[i], sh.B, sh.Hq, sh.N)) return false;
    for (int i = 0; i < nk; ++i)
        if (!rows_fit(k_side[i], sh.B, sh.Hk, sh.M)) return false;
    return true;
}

size_t tc_workspace(const Shape &sh, int sms, bool backward) {
    const size_t part = up(sizeof(int4) * (size_t)sms) +
                        up(sizeof(float) * 2 * (size_t)sms * (sh.state() + sh.d));
    return backward ? part + up(sizeof(float) * (size_t)(sh.heads() * sh.state())) +
                          up(sizeof(float) * (size_t)(sh.heads() * sh.d))
                    : part;
}

cudaError_t tc_state(const Shape &sh, Rows k, Rows v, float *S, float *z, char *ws, int sms,
                     int *status, cudaStream_t s) {
    return sh.d <= 64 ? state<64>(sh, k, v, S, z, ws, sms, status, s)
                      : state<128>(sh, k, v, S, z, ws, sms, status, s);
}

cudaError_t tc_read(const Shape &sh, Rows q, Rows out, const float *S, const float *z,
                    bool dependent, int sms, int *status, cudaStream_t s) {
    return sh.d <= 64 ? read<64>(sh, q, out, S, z, dependent, sms, status, s)
                      : read<128>(sh, q, out, S, z, dependent, sms, status, s);
}

cudaError_t tc_backward(const Shape &sh, Rows dout, Rows q, Rows k, Rows v, const float *S,
                        const float *z, Rows dq, Rows dk, Rows dv, char *ws, int sms, int *status,
                        cudaStream_t s) {
    return sh.d <= 64 ? back<64>(sh, dout, q, k, v, S, z, dq, dk, dv, ws, sms, status, s)
                      : back<128>(sh, dout, q, k, v, S, z, dq, dk, dv, ws, sms, status, s);
}

}  // namespace cross
}  // namespace la

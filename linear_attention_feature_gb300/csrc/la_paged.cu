// Softmax attention of new tokens over a paged cache (la_decode_step_paged in
// include/linattn.h):
//   o_t = sum_j exp(s_tj) v_j / sum_j exp(s_tj),  s_tj = scale q_t . k_j,
// over the keys j in (p_t - window, p_t], p_t = lengths[b] + t.
//
// One pass over keys and values: each warp keeps the running maximum m, the sum l
// of exp(s - m) and the output times l, all fp32, and multiplies the last two by
// exp(m_old - m_new) where the maximum moves.  Bound by reading the cache.
//
// The split.  The call's work is one list: for each sequence, head of keys and tile
// of queries the tiles of kTile keys that it looks at.  Every block finds the list's
// length from `lengths` itself and takes an equal piece, whatever the sequences'
// lengths.  A stretch of tiles with the same queries that lies in one block is
// written at once; what lies in several leaves (m, l, output) of each piece in the
// workspace, and a second kernel joins the pieces in order.  Repeated calls are
// bit-identical.
//
// Measured, bf16, join included: 32 heads on 8 of 128, 1 x 131072 keys 93 us, 5.8 TB/s;
// 256 x up to 4096 keys 397 us, 6.3 TB/s; 4 new tokens, 16 heads of 64, against 32 x up to
// 8192 keys 119 us, 5.6 TB/s.  A call takes 10 to 14 us more than its bytes:
// the way to the first keys (lengths, table, tile: one after the other), the pieces'
// unequal ends, the join.  Small calls take 7 to 18 us, whatever they read.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "la_internal.h"
#include "la_layer.cuh"
#include "la_tc.h"
#include "la_tc_common.cuh"
#include "la_tc_host.h"
#include "la_tc_ptx.cuh"

namespace la {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMostTokens = 1 << 30, kMostNew = 1 << 20;  // of a sequence, of a call
constexpr int kRowTile = 16;  // queries of one head of keys that a block takes at most

struct Params {
    const void *q, *k, *v;
    void *out;
    la_strides sq, so, sk, sv;
    const int *table, *lengths;
    long long table_stride;
    int pages, page_size, max_pages, page_shift;  // page_size is 2^page_shift, or -1
    int B, Hk, G, T, d, window;
    int *status;
    int q_words;     // queries lie in 32-bit words
    int row_tile, row_tiles;  // queries of a block, tiles of them per head of keys
    float scale2;             // scale log2(e)
    int4 *info;               // of each block: see Plan
    float *part;              // [blocks][2][row_tile][d + 2]
    long long timeout;        // clock cycles per wait
    int hold;                 // test hook: warps fetch no tile from this one of their own on, or -1
};

// Where a sequence's keys lie: [lo, hi) in tiles of kTile from the one of lo on.  One
// that takes no keys (an unused place in the batch) has one tile, all masked, so that
// its zeros get written.
struct Span {
    int before, lo, hi, first, tiles;
    int reach;  // query t looks at keys above before + t - reach
};

template <int kTile>
__device__ __forceinline__ Span span_of(const Params &p, int b) {
    Span s;
    // Beyond all that a table can hold, queries look at its last keys from nearer by: the
    // window is as much shorter.
    const int length = p.lengths[b];
    s.before = min(length, kMostTokens);
    s.hi = s.before < 0 ? 0 : min(s.before + p.T, p.max_pages * p.page_size);
    // the key before those of the first query; -kMostNew: none is before any query's
    const int low = p.window > 0 ? (int)min(max((long long)length - p.window, -(long long)kMostNew),
                                            (long long)kMostTokens)
                                 : -kMostNew;
    s.lo = min(max(low + 1, 0), s.hi);
    s.reach = s.before - low;
    s.first = s.lo / kTile;
    s.tiles = max(1, (s.hi + kTile - 1) / kTile - s.first);
    return s;
}

// Whether all queries of the call look at all of n keys from key0 on.
__device__ __forceinline__ bool all_see(const Params &p, const Span &s, int key0, int n) {
    return key0 + n - 1 <= s.before && key0 > s.before + p.T - 1 - s.reach;
}

// A place in the list of tiles.
template <int kTile>
struct Place {
    Span s;
    int b, seg, tile;  // seg: head of keys and tile of queries

    __device__ __forceinline__ void next(const Params &p, int segs) {
        if (++tile < s.tiles) return;
        tile = 0;
        if (++seg < segs) return;
        seg = 0;
        if (++b < p.B) s = span_of<kTile>(p, b);
    }
};

// This block's piece of the list and the place of its first tile.
template <int kTile>
__device__ __forceinline__ Place<kTile> find_place(const Params &p, long long *shared,
                                                   Piece &piece) {
    piece = find_piece<kThreads>(
        p.B, p.Hk * p.row_tiles, 1, [&](int b) { return span_of<kTile>(p, b).tiles; }, shared);
    Place<kTile> c;
    c.b = piece.b;
    if (piece.x0 < piece.x1) {
        c.s = span_of<kTile>(p, c.b);
        c.seg = (int)(piece.rest <= 0x7fffffff ? (unsigned)piece.rest / (unsigned)c.s.tiles
                                               : piece.rest / c.s.tiles);
        c.tile = (int)(piece.rest - (long long)c.seg * c.s.tiles);
    }
    return c;
}

// One (m, l) pair of running statistics and its merge: the factor of what went before.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ void copy16(unsigned dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(unsigned dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 4 : 0) : "memory");
}

// Copies kKeys rows of keys and of values into one stage of a warp's ring.  Lane l <
// kKeys holds where row l lies (offsets in elements) and whether it is to be read; the
// others are filled with zeros.  kUnit: bytes of a copy; 2: plain loads.
template <typename T, int kD, int kPitch, int kKeys, int kUnit>
__device__ __forceinline__ void copy_rows(const Params &p, T *stage, long long ko, long long vo,
                                          bool ok) {
    const int lane = threadIdx.x & 31;
    const T *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
    const int units = p.d * (int)sizeof(T) / kUnit;
    constexpr int kPer = kUnit / (int)sizeof(T);  // elements
    constexpr int kMost = kD / kPer;
    constexpr int kLanes = kUnit < 16 || kMost > 16 ? 32 : kMost > 8 ? 16 : kMost > 4 ? 8 : 4;
#pragma unroll
    for (int r = 0; r < kKeys; r += 32 / kLanes) {
        const int row = r + lane / kLanes;
        const long long kr = __shfl_sync(~0u, ko, row), vr = __shfl_sync(~0u, vo, row);
        const bool fine = __shfl_sync(~0u, (int)ok, row);
        const unsigned dst = tc::smem_u32(stage + row * kPitch);
        constexpr unsigned kOther = kKeys * kPitch * sizeof(T);
        for (int u = lane % kLanes; u < units; u += kLanes) {
            const T *ks = fine ? k + kr + u * kPer : k, *vs = fine ? v + vr + u * kPer : v;
            if constexpr (kUnit == 16) {
                copy16(dst + u * 16, ks, fine);
                copy16(dst + kOther + u * 16, vs, fine);
            } else if constexpr (kUnit == 4) {
                copy4(dst + u * 4, ks, fine);
                copy4(dst + kOther + u * 4, vs, fine);
            } else {
                stage[row * kPitch + u] = fine ? *ks : T(0.f);
                stage[(kKeys + row) * kPitch + u] = fine ? *vs : T(0.f);
            }
        }
    }
}

// Where a key lies: the page that the table names and the slot in it.
struct Slot {
    int key, page, slot;
};

template <int kTile, int kKeys>
__device__ __forceinline__ Slot slot_of(const Params &p, const Place<kTile> &c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Slot s;
    s.key = (c.s.first + c.tile) * kTile + warp * kKeys + lane;
    s.page = -1;
    s.slot = 0;
    if (lane < kKeys && s.key >= c.s.lo && s.key < c.s.hi) {
        const int column = s.key / p.page_size;
        s.slot = s.key - column * p.page_size;
        s.page = p.table[c.b * p.table_stride + column];
        if (s.page >= p.pages) s.page = -1;
    }
    return s;
}

// The same of a warp's whole tile, where pages hold whole tiles: the first key, whatever
// the bounds are.
template <int kTile, int kKeys>
__device__ __forceinline__ Slot tile_of(const Params &p, const Place<kTile> &c) {
    Slot s;
    s.key = (c.s.first + c.tile) * kTile + (threadIdx.x >> 5) * kKeys;
    s.page = -1;
    const int column = p.page_shift >= 0 ? s.key >> p.page_shift : s.key / p.page_size;
    s.slot = s.key - column * p.page_size;
    if (s.key < c.s.hi && s.key + kKeys > c.s.lo) {
        s.page = __ldg(p.table + c.b * p.table_stride + column);
        if (s.page >= p.pages) s.page = -1;
    }
    return s;
}

// Output rows of a block: the queries of one tile.  Row r of the head's G T queries is
// query t = r % T of head r / T of the group.
template <typename T>
__device__ __forceinline__ long long row_offset(const Params &p, const la_strides &s, int b, int h,
                                                int r) {
    const int g = r / p.T, t = r - g * p.T;
    return b * s.b + (long long)(h * p.G + g) * s.h + t * s.n;
}

// One value of a finished stretch, or of one that is left for the join (slot >= 0): the
// output y times l, the maximum and l.
template <typename T>
__device__ __forceinline__ void write_value(const Params &p, int b, int h, int row0, int r, int c,
                                            int slot, float y, float m, float l) {
    if (slot < 0) {
        T *out = static_cast<T *>(p.out) + row_offset<T>(p, p.so, b, h, row0 + r);
        from_f(out[c], l == 0.f ? 0.f : y / l);
    } else {
        float *w = p.part + ((long long)(blockIdx.x * 2 + slot) * p.row_tile + r) * (p.d + 2);
        w[c] = y;
        if (c == 0) w[p.d] = m, w[p.d + 1] = l;
    }
}

// What the join has to know of each block: the stretch that its piece continues (b segs +
// seg, 64 bits: .x low, .y high; .y = -1: none) and the first and the last block that have
// pieces of it (.z, .w).
__device__ __forceinline__ void note(const Params &p, long long stretch, int i0, int i1) {
    p.info[blockIdx.x] = make_int4((int)(unsigned)stretch, (int)(stretch >> 32), i0, i1);
}

// ------------------------------------------------------------------ bf16

__device__ __forceinline__ void ldmatrix4(unsigned (&r)[4], unsigned at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(unsigned (&r)[4], unsigned at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// c += a b, 16 x 16 times 16 x 8.
__device__ __forceinline__ void mma(float (&c)[4], const unsigned (&a)[4], unsigned b0,
                                    unsigned b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// kUnit: bytes of a copy (4 or 16 with cp.async, 2 with plain loads, rows kPitch apart in
// shared memory), or 0: tiles by TMA, in atoms of 64 features with the 128-byte swizzle.
template <int kD, int kUnit>
struct Half {
    static constexpr int kKeys = 16, kTile = kWarps * kKeys;
    static constexpr int kPitch = kD + 8;  // 16 bytes more than the row: no bank conflicts
    static constexpr int kSide = kUnit ? kKeys * kPitch * 2 : kKeys * kD * 2;  // keys, or values
    static constexpr int kStage = 2 * kSide;                                   // of a warp
    static constexpr int kStages = kD == 64 || kD == 192 ? 4 : 3;
    static constexpr int kBlocks = kD == 64 && kUnit == 0 ? 3 : kD <= 128 ? 2 : 1;  // per SM
    // Steps of the products' 16 features whose queries lie in registers; the rest of
    // them, which would spill, in each lane's 16 bytes of shared memory.
    static constexpr int kHeld = kD <= 128 ? kD / 16 : kD == 192 ? 8 : 6, kOffQ = kWarps * kStages * kStage;
    static constexpr int kOffMl = kOffQ + kWarps * (kD / 16 - kHeld) * 512;
    static constexpr int kOffMask = kOffMl + kWarps * kRowTile * 8;
    static constexpr int kOffBar = kOffMask + kWarps * kStages * 4;
    static_assert(kRowTile * kD * 4 <= kStage, "a warp's outputs fit into a stage");
    static constexpr int kOffPlan = kOffBar + kWarps * kStages * 8;
    static constexpr int kSmem = kOffPlan + (kWarps + 2) * 8 + 16 + (kUnit ? 0 : 1024);
    static_assert(kOffBar % 8 == 0 && kSmem <= 232448, "shared memory");
    static_assert(kSmem + 1024 <= 233472 / kBlocks, "blocks per SM");
};

// Rows of one side of the cache as a TMA tensor [page][head][slot][feature].
__device__ __forceinline__ void load_keys(unsigned dst, const CUtensorMap *map, uint64_t *bar,
                                          int c, int slot, int h, int page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(map), "r"(c), "r"(slot), "r"(h),
        "r"(page), "r"(tc::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 queries of one head of keys (the heads that share it, and the call's tokens)
// against 16 keys per warp and step: m16n8k16 products, whose 16 rows would be empty
// for one query, but the tensor cores wait for the memory all the same.  P is rounded
// to bf16 for its product with the values; l sums the rounded ones (a product with a
// column of ones), so that the weights still add to one.
//
// Each warp has its own ring of stages, so no warp waits for another before the stretch's
// end.  32 sequences of up to 8192 keys (4096 with d = 256), 4 heads shared by 4 each: d =
// 64 39 us, 128 65 us, 256 96 us (102 us with all queries in registers, which spills).
// Sums in two chains per score change nothing: the products are not what it waits for.
template <int kD, int kUnit>
__global__ void __launch_bounds__(kThreads, Half<kD, kUnit>::kBlocks)
paged_half_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv) {
    using L = Half<kD, kUnit>;
    using T = __nv_bfloat16;
    constexpr int kTile = L::kTile, kKeys = L::kKeys;
    constexpr unsigned kAtom = kUnit ? 128 : kKeys * 128;  // bytes from 64 features to the next
    extern __shared__ __align__(128) char raw[];
    char *smem = kUnit ? raw
                       : reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                  ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    char *ring = smem + warp * L::kStages * L::kStage;
    float2 *ml = reinterpret_cast<float2 *>(smem + L::kOffMl);
    unsigned *masks = reinterpret_cast<unsigned *>(smem + L::kOffMask) + warp * L::kStages;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar) + warp * L::kStages;
    int *abort = reinterpret_cast<int *>(smem + L::kOffPlan + (kWarps + 2) * 8);
    const tcc::Ctx cx{abort, p.status, p.timeout};
    const int segs = p.Hk * p.row_tiles;

    if (kUnit != 0)  // features from d on
        for (int i = threadIdx.x; i < L::kOffMl / 16; i += kThreads)
            reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) *abort = 0;
    if (kUnit == 0) {
        if (lane == 0) {
            for (int i = 0; i < L::kStages; ++i) tc::mbar_init(bars + i, 1);
            tc::fence_mbar_init();
        }
        tc::fence_async_shared();
    }
    Piece piece;
    Place<kTile> c =
        find_place<kTile>(p, reinterpret_cast<long long *>(smem + L::kOffPlan), piece);
    if (threadIdx.x == 0) note(p, -1, 0, 0);
    const long long x1 = piece.x1;
    const int steps = (int)(x1 - piece.x0);
    if (steps == 0) return;

    // the copying side, some tiles ahead; `ahead` is where the next tile's keys lie
    Place<kTile> f = c;
    int f_left = steps, f_stage = 0;
    Slot ahead;
    auto look = [&]() {
        if constexpr (kUnit)
            ahead = slot_of<kTile, kKeys>(p, f);
        else
            ahead = tile_of<kTile, kKeys>(p, f);
    };
    look();
    auto fetch = [&]() {
        if (f_left > 0) {
            const int h = p.row_tiles == 1 ? f.seg : f.seg / p.row_tiles;
            char *stage = ring + f_stage * L::kStage;
            unsigned mask;
            if constexpr (kUnit) {
                const bool ok = ahead.page >= 0;
                copy_rows<T, kD, L::kPitch, kKeys, kUnit ? kUnit : 16>(
                    p, reinterpret_cast<T *>(stage),
                    ahead.page * p.sk.b + h * p.sk.h + ahead.slot * p.sk.n,
                    ahead.page * p.sv.b + h * p.sv.h + ahead.slot * p.sv.n, ok);
                mask = __ballot_sync(~0u, ok);
            } else {
                // the tile's keys are in one page
                const int first = max(f.s.lo - ahead.key, 0), n = min(f.s.hi - ahead.key, kKeys);
                mask = ahead.page >= 0 && n > first ? (0xffffu >> (kKeys - n)) >> first << first : 0;
                if (lane == 0 && steps - f_left != p.hold) {
                    if (mask == 0) {
                        tc::mbar_arrive(bars + f_stage);
                    } else {
                        const int atoms = (p.d + 63) / 64;
                        tc::mbar_arrive_expect_tx(bars + f_stage, atoms * 2 * kKeys * 128);
                        for (int a = 0; a < atoms; ++a) {
                            const unsigned at = tc::smem_u32(stage) + a * kAtom;
                            load_keys(at, &tk, bars + f_stage, 64 * a, ahead.slot, h, ahead.page);
                            load_keys(at + L::kSide, &tv, bars + f_stage, 64 * a, ahead.slot, h,
                                      ahead.page);
                        }
                    }
                }
            }
            if (lane == 0) masks[f_stage] = mask;
            f_stage = f_stage + 1 == L::kStages ? 0 : f_stage + 1;
            if (--f_left > 0) {
                f.next(p, segs);
                look();
            }
        }
        if constexpr (kUnit != 0) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < L::kStages - 1; ++i) fetch();

    // where a lane's rows for ldmatrix lie: 16 features further on, and 64
    unsigned k_at[4], v_at[4];
    {
        const int kr = (lane & 7) + (lane >> 4) * 8, vr = lane & 15;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int kc = 2 * i + ((lane >> 3) & 1), vc = 2 * i + (lane >> 4);
            k_at[i] = kUnit ? kr * L::kPitch * 2 + kc * 16 : kr * 128 + (kc ^ (kr & 7)) * 16;
            v_at[i] = kUnit ? vr * L::kPitch * 2 + vc * 16 : vr * 128 + (vc ^ (vr & 7)) * 16;
            v_at[i] += L::kSide;
        }
    }
    // The queries as the products take them, straight from memory: rows lane / 4 and 8
    // further on, features 2 (lane % 4) and 8 further on of each 16.
    unsigned a[L::kHeld][4];
    uint4 *rest = reinterpret_cast<uint4 *>(smem + L::kOffQ) + warp * (kD / 16 - L::kHeld) * 32 + lane;
    auto load_queries = [&]() {
        const int h = c.seg / p.row_tiles, row0 = (c.seg - h * p.row_tiles) * p.row_tile;
        const int rows = min(p.row_tile, p.G * p.T - row0);
        const T *q[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (lane >> 2) + 8 * i;
            q[i] = static_cast<const T *>(p.q) +
                   (r < rows ? row_offset<T>(p, p.sq, c.b, h, row0 + r) : 0);
        }
        auto load_step = [&](int ks, unsigned (&to)[4]) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = (lane >> 2) + 8 * i;
                    const int e = 16 * ks + 8 * j + 2 * (lane & 3);
                    unsigned u = 0;
                    if (r < rows && e < p.d) {
                        if (p.q_words) {
                            u = *reinterpret_cast<const unsigned *>(q[i] + e);
                        } else {
                            u = *reinterpret_cast<const unsigned short *>(q[i] + e);
                            if (e + 1 < p.d)
                                u |= (unsigned)*reinterpret_cast<const unsigned short *>(q[i] + e + 1)
                                     << 16;
                        }
                    }
                    to[2 * j + i] = u;
                }
        };
#pragma unroll
        for (int ks = 0; ks < L::kHeld; ++ks) load_step(ks, a[ks]);
#pragma unroll 4
        for (int ks = L::kHeld; ks < kD / 16; ++ks) {
            unsigned u[4];
            load_step(ks, u);
            rest[(ks - L::kHeld) * 32] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    };
    load_queries();

    int stage = 0;
    unsigned parity = 0;
    for (int left = steps; left > 0;) {
        // ---- a stretch of tiles with the same queries
        const int h = c.seg / p.row_tiles, row0 = (c.seg - h * p.row_tiles) * p.row_tile;
        const int rows = min(p.row_tile, p.G * p.T - row0);
        const bool began = c.tile > 0;  // in an earlier block
        const long long x = x1 - left;
        const long long seg0 = x - c.tile, seg1 = seg0 + c.s.tiles;
        const int n = (int)min((long long)left, seg1 - x);
        float o[kD / 8][4], sums[4] = {};  // the outputs times l, and l
#pragma unroll
        for (int j = 0; j < kD / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY};
        // A wait has run out: nothing more is fetched, since a barrier must not be armed again
        // while its copy is under way, and what is under way lands.
        auto give_up = [&](int it) {
            if (f_left < 0) return;  // all that has been fetched is there
            for (int i = steps - left + it; i < steps - f_left; ++i)
                if (i != p.hold) tcc::settle_wait(bars + i % L::kStages, i / L::kStages & 1);
            f_left = -1;
        };
        // the last key of this lane's two queries
        int last[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            last[i] = c.s.before + (row0 + (lane >> 2) + 8 * i) % p.T;

        for (int it = 0; it < n; ++it) {
            fetch();
            if constexpr (kUnit != 0)
                asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 1) : "memory");
            else if (!tcc::wait_bar(bars + stage, parity, cx))
                give_up(it);
            __syncwarp();
            const unsigned st = tc::smem_u32(ring + stage * L::kStage);
            T *values = reinterpret_cast<T *>(ring + stage * L::kStage + L::kSide);
            const unsigned mask = masks[stage];
            const int key0 = (c.s.first + c.tile) * kTile + warp * kKeys;
            float s[2][4] = {};
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                unsigned b[4];
                ldmatrix4(b, st + k_at[ks & 3] + (ks >> 2) * kAtom);
                unsigned w[4];
                if (ks < L::kHeld) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = a[ks < L::kHeld ? ks : 0][i];
                } else {
                    const uint4 u = rest[(ks - L::kHeld) * 32];
                    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
                }
                mma(s[0], w, b[0], b[1]);
                mma(s[1], w, b[2], b[3]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j][e] *= p.scale2;
            const bool whole = mask == 0xffffu && all_see(p, c.s, key0, kKeys);
            // A weight of 0 does not keep a value that is not finite out of a sum: slots
            // that hold no key of the sequence become 0, and a tile where queries look at
            // different keys takes values that are not finite singly.
            bool singly = false;
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = j * 8 + (lane & 3) * 2 + (e & 1), key = key0 + i;
                        const int end = last[e >> 1];
                        if (!(mask >> i & 1) || key > end || key <= end - c.s.reach)
                            s[j][e] = -INFINITY;
                    }
                if (kUnit == 0 && mask != 0xffffu) {
                    for (int i = 0; i < kKeys; ++i)
                        if (!(mask >> i & 1))
                            for (int q = 0; q < kD / 64; ++q)
                                reinterpret_cast<unsigned *>(values)[(q * kAtom + i * 128) / 4 +
                                                                     lane] = 0;
                    tc::fence_async_shared();  // before the next tile arrives here
                    __syncwarp();
                }
                if (p.T > 1) {
                    bool odd = false;
                    for (int i = lane; i < L::kSide / 2; i += 32)
                        odd |= (kUnit == 0 || i % L::kPitch < kD) &&
                               !(fabsf(to_f(values[i])) < INFINITY);
                    singly = __any_sync(~0u, odd);
                }
            }
            float top[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]),
                               fmaxf(s[1][2 * i], s[1][2 * i + 1]));
                top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], 2));
                top[i] = fmaxf(top[i], m[i]);
            }
            if (__any_sync(~0u, top[0] > m[0] || top[1] > m[1])) {
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[i] = exp2_fast(m[i] - finite_max(top[i]));
                    m[i] = top[i];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) sums[e] *= w[e >> 1];
#pragma unroll
                for (int j = 0; j < kD / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][e] *= w[e >> 1];
            }
            unsigned pa[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mi = finite_max(m[i]);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    pa[2 * j + i] = tc::pack_bf16x2(exp2_fast(s[j][2 * i] - mi),
                                                    exp2_fast(s[j][2 * i + 1] - mi));
            }
            mma(sums, pa, 0x3F803F80u, 0x3F803F80u);
            if (singly) {
                for (int i = 0; i < kKeys; ++i) {
                    const int from = (lane & 28) + (i & 7) / 2;
                    unsigned u[2];  // of the two queries
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const unsigned lo = __shfl_sync(~0u, pa[r], from);
                        const unsigned hi = __shfl_sync(~0u, pa[2 + r], from);
                        u[r] = i < 8 ? lo : hi;
                        u[r] = i & 1 ? u[r] & 0xffff0000u : u[r] << 16;
                    }
#pragma unroll
                    for (int j = 0; j < kD / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int col = 8 * j + (lane & 3) * 2 + (e & 1);
                            const unsigned at =
                                kUnit ? i * L::kPitch * 2 + col * 2
                                      : (col >> 6) * kAtom + tc::sw128_offset(i, col & 63);
                            if (u[e >> 1])
                                o[j][e] = fmaf(__uint_as_float(u[e >> 1]), to_f(values[at / 2]),
                                               o[j][e]);
                        }
                }
            } else {
#pragma unroll
                for (int j = 0; j < kD / 16; ++j) {
                    unsigned b[4];
                    ldmatrix4_t(b, st + v_at[j & 3] + (j >> 2) * kAtom);
                    mma(o[2 * j], pa, b[0], b[1]);
                    mma(o[2 * j + 1], pa, b[2], b[3]);
                }
            }
            __syncwarp();  // the stage may be filled again
            if (++stage == L::kStages) stage = 0, parity ^= 1;
            c.tile += 1;
        }
        // ---- the warps' parts together, through the places that they have just read; the
        // next stretch's queries come meanwhile
        const int b = c.b, seg = c.seg;
        left -= n;
        c.tile -= 1;
        if (left > 0) {
            c.next(p, segs);
            load_queries();
        }
        const int mine = stage == 0 ? L::kStages - 1 : stage - 1;
        auto place = [&](int q) {
            return reinterpret_cast<float *>(smem + (q * L::kStages + mine) * L::kStage);
        };
        // (columns turned by 8 per row: no bank conflicts)
        auto at = [](int r, int col) { return r * kD + (col ^ (r & 3) << 3); };
#pragma unroll
        for (int j = 0; j < kD / 8; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float2 *>(
                    place(warp) + at((lane >> 2) + 8 * i, 8 * j + (lane & 3) * 2)) =
                    make_float2(o[j][2 * i], o[j][2 * i + 1]);
        if ((lane & 3) == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                ml[warp * kRowTile + (lane >> 2) + 8 * i] = make_float2(m[i], sums[2 * i]);
        __syncthreads();
        const bool ends = seg1 <= x1;
        const int slot = began ? 0 : ends ? -1 : 1;
        for (int i = threadIdx.x; i < rows * p.d; i += kThreads) {
            const int r = i / p.d, col = i - r * p.d;
            float top = -INFINITY, sum = 0.f, y = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) top = fmaxf(top, ml[q * kRowTile + r].x);
#pragma unroll
            for (int q = 0; q < kWarps; ++q) {
                const float2 v = ml[q * kRowTile + r];
                const float w = exp2_fast(v.x - finite_max(top));
                sum = fmaf(v.y, w, sum);
                y = fmaf(place(q)[at(r, col)], w, y);
            }
            write_value<T>(p, b, h, row0, r, col, slot, y, top, sum);
        }
        if (began && threadIdx.x == 0)
            note(p, (long long)b * segs + seg, piece.of(seg0), piece.of(seg1 - 1));
        if (kUnit == 0) tc::fence_async_shared();  // before the next tile arrives there
        __syncthreads();
        if (kUnit != 0 && p.d < kD) {  // features from d on are 0 again
            for (int i = lane; i < L::kStage / 16; i += 32)
                reinterpret_cast<uint4 *>(place(warp))[i] = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
    }
    if constexpr (kUnit != 0) asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ fp32

template <int kD>
struct Full {
    static constexpr int kKeys = kD == 64 ? 16 : 8, kTile = kWarps * kKeys;
    static constexpr int kParts = 32 / kKeys;  // lanes that share a key
    static constexpr int kPitch = kD + 4;
    static constexpr int kStage = 2 * kKeys * kPitch * 4;
    static constexpr int kStages = 3;
    static constexpr int kBlocks = kD <= 128 ? 2 : 1;
    static constexpr int kOffQ = kWarps * kStages * kStage;  // then the output
    static constexpr int kOffP = kOffQ + 8 * kPitch * 4;     // [warp][row][key]
    static constexpr int kOffMl = kOffP + kWarps * 8 * kKeys * 4;
    static constexpr int kOffMask = kOffMl + (kWarps + 1) * 8 * 8;
    static constexpr int kOffPlan = kOffMask + kWarps * kStages * 4;
    static constexpr int kSmem = kOffPlan + (kWarps + 2) * 8;
    static_assert(kOffPlan % 8 == 0 && kSmem <= 232448, "shared memory");
    static_assert(kSmem + 1024 <= 233472 / kBlocks, "blocks per SM");
};

// kR queries per block.  A warp takes kKeys keys per step: kParts lanes share a key's
// scores, each with every kParts-th 16 bytes of it; then each lane takes every 32nd
// feature of the values.  fp32 throughout.  The case above with d = 128: 169 us with 4
// queries per key (4.0 TB/s), 133 us with one (5.0 TB/s); bound by the latency of a warp's
// step, 8 warps per SM.  (A running maximum per query, each with its branch, and features
// counted up to d: 192 us.  Queries in registers, where they fit: 166 us.)
template <int kD, int kR, int kUnit>
__global__ void __launch_bounds__(kThreads, Full<kD>::kBlocks)
paged_full_kernel(const __grid_constant__ Params p) {
    using L = Full<kD>;
    using T = float;
    constexpr int kTile = L::kTile, kKeys = L::kKeys, kCols = kD / 32;
    extern __shared__ __align__(128) char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    char *ring = smem + warp * L::kStages * L::kStage;
    float *qbuf = reinterpret_cast<float *>(smem + L::kOffQ);
    float *pbuf = reinterpret_cast<float *>(smem + L::kOffP) + warp * 8 * kKeys;
    float2 *ml = reinterpret_cast<float2 *>(smem + L::kOffMl);
    unsigned *masks = reinterpret_cast<unsigned *>(smem + L::kOffMask) + warp * L::kStages;
    const int segs = p.Hk * p.row_tiles;

    for (int i = threadIdx.x; i < L::kOffQ / 16; i += kThreads)
        reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
    Piece piece;
    Place<kTile> c =
        find_place<kTile>(p, reinterpret_cast<long long *>(smem + L::kOffPlan), piece);
    if (threadIdx.x == 0) note(p, -1, 0, 0);
    const long long x1 = piece.x1;
    const int steps = (int)(x1 - piece.x0);
    if (steps == 0) return;

    Place<kTile> f = c;
    int f_left = steps, f_stage = 0;
    Slot ahead = slot_of<kTile, kKeys>(p, f);
    auto fetch = [&]() {
        if (f_left > 0) {
            const int h = f.seg / p.row_tiles;
            const bool ok = ahead.page >= 0;
            copy_rows<T, kD, L::kPitch, kKeys, kUnit>(
                p, reinterpret_cast<T *>(ring + f_stage * L::kStage),
                ahead.page * p.sk.b + h * p.sk.h + ahead.slot * p.sk.n,
                ahead.page * p.sv.b + h * p.sv.h + ahead.slot * p.sv.n, ok);
            const unsigned mask = __ballot_sync(~0u, ok);
            if (lane == 0) masks[f_stage] = mask;
            f_stage = f_stage + 1 == L::kStages ? 0 : f_stage + 1;
            if (--f_left > 0) {
                f.next(p, segs);
                ahead = slot_of<kTile, kKeys>(p, f);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < L::kStages - 1; ++i) fetch();

    const int key_in = lane % kKeys, part = lane / kKeys;
    int stage = 0;
    for (int left = steps; left > 0;) {
        const int h = c.seg / p.row_tiles, row0 = (c.seg - h * p.row_tiles) * p.row_tile;
        const int rows = min(p.row_tile, p.G * p.T - row0);
        const bool began = c.tile > 0;
        const long long x = x1 - left;
        const long long seg0 = x - c.tile, seg1 = seg0 + c.s.tiles;
        const int n = (int)min((long long)left, seg1 - x);
        for (int i = threadIdx.x; i < kR * kD; i += kThreads) {
            const int r = i / kD, e = i % kD;
            float value = 0.f;
            if (r < rows && e < p.d)
                value = static_cast<const float *>(
                    p.q)[row_offset<T>(p, p.sq, c.b, h, row0 + r) + e];
            qbuf[r * L::kPitch + e] = value;
        }
        __syncthreads();
        float o[kR][kCols] = {}, m[kR], l[kR];
        int last[kR];  // the last key of each query
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            m[r] = -INFINITY, l[r] = 0.f;
            last[r] = c.s.before + (row0 + r) % p.T;
        }

        for (int it = 0; it < n; ++it) {
            fetch();
            asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 1) : "memory");
            __syncwarp();
            const float *ks = reinterpret_cast<const float *>(ring + stage * L::kStage);
            const float *vs = ks + kKeys * L::kPitch;
            const unsigned mask = masks[stage];
            const int key = (c.s.first + c.tile) * kTile + warp * kKeys + key_in;
            const bool whole = all_see(p, c.s, key - key_in, kKeys);
            float s[kR] = {};
#pragma unroll
            for (int i = 0; i < kD; i += 4 * L::kParts) {
                const int e = i + 4 * part;  // (features from d on are 0)
                if (i >= p.d) break;
                const float4 k4 = *reinterpret_cast<const float4 *>(ks + key_in * L::kPitch + e);
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const float4 q4 =
                        *reinterpret_cast<const float4 *>(qbuf + r * L::kPitch + e);
                    s[r] = fmaf(q4.x, k4.x, s[r]);
                    s[r] = fmaf(q4.y, k4.y, s[r]);
                    s[r] = fmaf(q4.z, k4.z, s[r]);
                    s[r] = fmaf(q4.w, k4.w, s[r]);
                }
            }
            float top[kR];
            bool moved = false;  // the same in all lanes
#pragma unroll
            for (int r = 0; r < kR; ++r) {
#pragma unroll
                for (int w = kKeys; w < 32; w <<= 1) s[r] += __shfl_xor_sync(~0u, s[r], w);
                s[r] *= p.scale2;
                if (!(mask >> key_in & 1) || key > last[r] || key <= last[r] - c.s.reach)
                    s[r] = -INFINITY;
                top[r] = s[r];
#pragma unroll
                for (int w = 1; w < kKeys; w <<= 1)
                    top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], w));
                moved |= top[r] > m[r];
            }
            if (moved)
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const float t = fmaxf(top[r], m[r]), w = exp2f(m[r] - finite_max(t));
                    l[r] *= w;
#pragma unroll
                    for (int j = 0; j < kCols; ++j) o[r][j] *= w;
                    m[r] = t;
                }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const float w = exp2f(s[r] - finite_max(m[r]));
                if (part == 0) {
                    l[r] += w;
                    pbuf[r * kKeys + key_in] = w;
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kKeys; i += 4) {
                float4 w[kR];
#pragma unroll
                for (int r = 0; r < kR; ++r)
                    w[r] = *reinterpret_cast<const float4 *>(pbuf + r * kKeys + i);
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    const float *v0 = vs + i * L::kPitch + lane + 32 * j;
                    const float v[4] = {v0[0], v0[L::kPitch], v0[2 * L::kPitch],
                                        v0[3 * L::kPitch]};
                    if (!whole) {  // a key that one query looks at may not reach another
#pragma unroll
                        for (int r = 0; r < kR; ++r) {
                            if (w[r].x != 0.f) o[r][j] = fmaf(w[r].x, v[0], o[r][j]);
                            if (w[r].y != 0.f) o[r][j] = fmaf(w[r].y, v[1], o[r][j]);
                            if (w[r].z != 0.f) o[r][j] = fmaf(w[r].z, v[2], o[r][j]);
                            if (w[r].w != 0.f) o[r][j] = fmaf(w[r].w, v[3], o[r][j]);
                        }
                        continue;
                    }
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        o[r][j] = fmaf(w[r].x, v[0], o[r][j]);
                        o[r][j] = fmaf(w[r].y, v[1], o[r][j]);
                        o[r][j] = fmaf(w[r].z, v[2], o[r][j]);
                        o[r][j] = fmaf(w[r].w, v[3], o[r][j]);
                    }
                }
            }
            __syncwarp();
            stage = stage + 1 == L::kStages ? 0 : stage + 1;
            c.tile += 1;
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
#pragma unroll
            for (int w = 1; w < kKeys; w <<= 1) l[r] += __shfl_xor_sync(~0u, l[r], w);
            if (lane == 0) ml[warp * 8 + r] = make_float2(m[r], l[r]);
        }
        __syncthreads();
        float w[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) top = fmaxf(top, ml[q * 8 + r].x);
#pragma unroll
            for (int q = 0; q < kWarps; ++q)
                sum += ml[q * 8 + r].y * exp2f(ml[q * 8 + r].x - finite_max(top));
            w[r] = exp2f(m[r] - finite_max(top));
            if (threadIdx.x == 0) ml[kWarps * 8 + r] = make_float2(top, sum);
        }
        for (int q = 0; q < kWarps; ++q) {
            if (warp == q)
#pragma unroll
                for (int r = 0; r < kR; ++r)
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        float *y = qbuf + r * L::kPitch + lane + 32 * j;
                        *y = q > 0 ? *y + o[r][j] * w[r] : o[r][j] * w[r];
                    }
            __syncthreads();
        }
        const bool ends = seg1 <= x1;
        const int slot = began ? 0 : ends ? -1 : 1;
        for (int i = threadIdx.x; i < rows * p.d; i += kThreads) {
            const int r = i / p.d, col = i - r * p.d;
            const float2 v = ml[kWarps * 8 + r];
            write_value<T>(p, c.b, h, row0, r, col, slot, qbuf[r * L::kPitch + col], v.x, v.y);
        }
        if (began && threadIdx.x == 0)
            note(p, (long long)c.b * segs + c.seg, piece.of(seg0), piece.of(seg1 - 1));
        __syncthreads();
        left -= n;
        c.tile -= 1;
        if (left > 0) c.next(p, segs);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Joins the stretches that lie in several blocks, one query of one stretch a block: the
// first of a stretch's blocks that continues it.
// Every warp finds the pieces' factors by itself, 32 at a time in its lanes; kJoin groups
// of threads take every kJoin-th piece of the output.
constexpr int kJoin = 4;

template <typename T>
__global__ void __launch_bounds__(kJoin *LA_MAX_D) paged_join_kernel(const __grid_constant__ Params p) {
    tc::grid_dep_wait();
    __shared__ float sum[kJoin][LA_MAX_D];
    const int r = blockIdx.y;
    const int4 info = p.info[blockIdx.x + 1];
    if (info.y < 0 || info.z != (int)blockIdx.x) return;
    const long long stretch = (long long)info.y << 32 | (unsigned)info.x;
    const int segs = p.Hk * p.row_tiles;
    const int b = (int)(stretch / segs), seg = (int)(stretch - (long long)b * segs);
    const int h = seg / p.row_tiles, row0 = (seg - h * p.row_tiles) * p.row_tile;
    if (row0 + r >= p.G * p.T) return;
    const int i0 = info.z, i1 = info.w, lane = threadIdx.x & 31;
    const int cols = blockDim.x / kJoin, e = threadIdx.x % cols, group = threadIdx.x / cols;
    auto part = [&](int q) {
        return p.part + ((long long)(2 * q + (q == i0)) * p.row_tile + r) * (p.d + 2);
    };
    float top = -INFINITY;
    for (int q = i0 + lane; q <= i1; q += 32) top = fmaxf(top, __ldcg(part(q) + p.d));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    top = finite_max(top);
    float y = 0.f, l = 0.f;
    for (int q0 = i0; q0 <= i1; q0 += 32) {
        float f = 0.f;
        if (q0 + lane <= i1) {
            const float *w = part(q0 + lane) + p.d;
            f = exp2f(__ldcg(w) - top);
            l = fmaf(__ldcg(w + 1), f, l);
        }
        const int n = min(32, i1 + 1 - q0);
#pragma unroll 8
        for (int q = 0; q < n; q += kJoin) {
            const float fq = __shfl_sync(~0u, f, (q + group) & 31);
            if (q + group < n && e < p.d) y = fmaf(__ldcg(part(q0 + q + group) + e), fq, y);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    if (e < p.d) sum[group][e] = y;
    __syncthreads();
    if (group > 0 || e >= p.d) return;
#pragma unroll
    for (int g = 1; g < kJoin; ++g) y += sum[g][e];
    T *out = static_cast<T *>(p.out) + row_offset<T>(p, p.so, b, h, row0 + r);
    from_f(out[e], l == 0.f ? 0.f : y / l);
}

struct Choice {
    const void *kern;
    int smem, tile, blocks_per_sm;
};

template <int kD, int kUnit>
Choice choose_half() {
    using L = Half<kD, kUnit>;
    return {reinterpret_cast<const void *>(&paged_half_kernel<kD, kUnit>), L::kSmem, L::kTile,
            L::kBlocks};
}
template <int kUnit>
Choice choose_half(int d) {
    if (d <= 64) return choose_half<64, kUnit>();
    if (d <= 128) return choose_half<128, kUnit>();
    if (d <= 192) return choose_half<192, kUnit>();
    return choose_half<256, kUnit>();
}

// One side of the cache for tiles of 16 slots and 64 features.
bool make_map(CUtensorMap *map, const void *x, const la_strides &s, const la_cache &c, int Hk,
              int d) {
    cudaError_t e;
    auto enc = tchost::encode_fn(&e);
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)c.page_size, (cuuint64_t)Hk,
                                (cuuint64_t)c.pages};
    const long long n = c.page_size > 1 ? s.n : d, h = Hk > 1 ? s.h : n, b = c.pages > 1 ? s.b : n;
    const cuuint64_t strides[3] = {(cuuint64_t)n * 2, (cuuint64_t)h * 2, (cuuint64_t)b * 2};
    const cuuint32_t box[4] = {64, 16, 1, 1}, one[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(x), dims, strides, box,
               one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <int kD, int kR, int kUnit>
Choice choose_full() {
    return {reinterpret_cast<const void *>(&paged_full_kernel<kD, kR, kUnit>), Full<kD>::kSmem,
            Full<kD>::kTile, Full<kD>::kBlocks};
}
template <int kD, int kUnit>
Choice choose_full(int row_tile) {
    if (row_tile <= 1) return choose_full<kD, 1, kUnit>();
    if (row_tile <= 2) return choose_full<kD, 2, kUnit>();
    if (row_tile <= 4) return choose_full<kD, 4, kUnit>();
    return choose_full<kD, 8, kUnit>();
}
template <int kUnit>
Choice choose_full(int d, int row_tile) {
    if (d <= 64) return choose_full<64, kUnit>(row_tile);
    if (d <= 128) return choose_full<128, kUnit>(row_tile);
    return choose_full<256, kUnit>(row_tile);
}

int row_tile_of(long long rows, la_dtype dtype) {
    const int most = dtype == LA_F32 ? 8 : kRowTile;
    return (int)std::min<long long>(rows, most);
}

int blocks_of(int sms) { return 3 * sms; }  // at most

// Bytes of the workspace: the blocks' notes, then their two parts.
size_t workspace_of(int blocks, int row_tile, int d) {
    return sizeof(int4) * (size_t)blocks +
           sizeof(float) * 2 * (size_t)blocks * row_tile * (d + 2);
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

__attribute__((visibility("default")))
la_status la_decode_step_paged(const void *q, void *out, const la_cache *cache,
                               const la_strides *strides, float scale, int window, int B, int Hq,
                               int Hk, int T, int d, la_dtype dtype, void *workspace,
                               size_t workspace_bytes, la_stream_t stream) {
    const char *who = "la_decode_step_paged";
    if (Hq < 0 || T < 0) return layer_fail(LA_ERR_INVALID_ARG, who, "negative Hq or T");
    la_status st = check_cache(who, cache, B, Hk, d, dtype);
    if (st != LA_OK) return st;
    if (!std::isfinite(scale)) return layer_fail(LA_ERR_INVALID_ARG, who, "scale must be finite");
    if (window < 0) return layer_fail(LA_ERR_INVALID_ARG, who, "negative window");
    if (Hk == 0 ? Hq != 0 : Hq % Hk != 0)
        return layer_fail(LA_ERR_INVALID_ARG, who, "Hq must be a multiple of Hk");
    if (B == 0 || T == 0 || Hq == 0) return LA_OK;
    if (!q || !out) return layer_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
    const uintptr_t elem = dtype == LA_F32 ? 4 : 2;
    if ((uintptr_t)q % elem || (uintptr_t)out % elem)
        return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
    Params p{};
    p.q = q;
    p.out = out;
    p.sq = strides ? strides[0] : contiguous(Hq, T, d);
    p.so = strides ? strides[1] : contiguous(Hq, T, d);
    if (negative(p.sq) || negative(p.so))
        return layer_fail(LA_ERR_INVALID_ARG, who, "negative stride");
    if (!rows_disjoint(p.so, B, Hq, T, d))
        return layer_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
    if (out == q || out == cache->k || out == cache->v)
        return layer_fail(LA_ERR_INVALID_ARG, who, "out aliases an input");
    const long long rows = (long long)(Hq / Hk) * T;
    p.row_tile = row_tile_of(rows, dtype);
    const long long row_tiles = (rows + p.row_tile - 1) / p.row_tile;
    if (T > kMostNew || rows > 0x7fffffff || Hk * row_tiles > 0x7fffffff)
        return layer_fail(LA_ERR_UNSUPPORTED, who, "too many queries");
    p.row_tiles = (int)row_tiles;
    p.k = cache->pages ? cache->k : q;  // without pages nothing is read
    p.v = cache->pages ? cache->v : q;
    p.sk = cache->k_strides;
    p.sv = cache->v_strides;
    p.table = cache->table;
    p.lengths = cache->lengths;
    p.table_stride = cache->table_stride;
    p.pages = cache->pages;
    p.page_size = cache->page_size;
    p.max_pages = cache->max_pages;
    p.B = B;
    p.Hk = Hk;
    p.G = Hq / Hk;
    p.T = T;
    p.d = d;
    p.window = window;
    p.scale2 = scale * 1.44269504088896341f;
    {
        unsigned long long words = (uintptr_t)q / 2 | (unsigned)d;
        if (B > 1) words |= (unsigned long long)p.sq.b;
        if (Hq > 1) words |= (unsigned long long)p.sq.h;
        if (T > 1) words |= (unsigned long long)p.sq.n;
        p.q_words = words % 2 == 0;
    }
    p.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (p.page_size == 1 << i) p.page_shift = i;

    // bytes per copy: 16, or 4, if every row of the cache is aligned to that
    unsigned long long all = (uintptr_t)p.k | (uintptr_t)p.v | (unsigned)d * elem;
    auto add = [&](const la_strides &s) {
        if (p.pages > 1) all |= (unsigned long long)s.b * elem;
        if (Hk > 1) all |= (unsigned long long)s.h * elem;
        if (p.page_size > 1) all |= (unsigned long long)s.n * elem;
    };
    add(p.sk);
    add(p.sv);
    Choice c;
    CUtensorMap maps[2] = {};
    // TMA: pages of whole tiles, rows in 16-byte units, no stride of 0 or of 2^38 and more
    auto fit = [&](const la_strides &s) {
        const long long most = 1LL << 38;
        return (p.pages <= 1 || (s.b >= 8 && s.b < most)) && (Hk <= 1 || (s.h >= 8 && s.h < most)) &&
               s.n >= 8 && s.n < most;
    };
    const bool tiles_fit = dtype == LA_BF16 && all % 16 == 0 && p.page_size % 16 == 0 &&
                           p.pages > 0 && fit(p.sk) && fit(p.sv) &&
                           make_map(&maps[0], p.k, p.sk, *cache, Hk, d) &&
                           make_map(&maps[1], p.v, p.sv, *cache, Hk, d);
    if (tiles_fit)
        c = choose_half<0>(d);  // d = 128, the case at paged_half_kernel: 65 us; 16-byte copies 80
                                // us, 4-byte 143 us, plain loads 482 us
    else if (dtype == LA_F32)  // 4-byte copies take 1.25 times as long
        c = all % 16 == 0 ? choose_full<16>(d, p.row_tile) : choose_full<4>(d, p.row_tile);
    else
        c = all % 16 == 0 ? choose_half<16>(d)
                          : all % 4 == 0 ? choose_half<4>(d) : choose_half<2>(d);

    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e == cudaSuccess) p.status = device_status_word(&e);
    if (e != cudaSuccess) return layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    // No more blocks than tiles that the table could hold.
    const long long cap = (long long)p.max_pages * p.page_size;
    const long long tiles = std::max(1LL, (cap + c.tile - 1) / c.tile + 1);
    const double list = (double)B * Hk * (double)row_tiles * (double)tiles;
    if (list > 1e11) return layer_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
    const int blocks = (int)std::min((double)c.blocks_per_sm * sms, list);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t need = workspace_of(blocks, p.row_tile, d);
    void *ws = workspace, *own = nullptr;
    if (ws) {
        if (workspace_bytes < need || (uintptr_t)ws % 16)
            return layer_fail(LA_ERR_INVALID_ARG, who,
                              "workspace too small or not 16-byte aligned");
    } else {
        e = tc_workspace_alloc(&own, need, s);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return layer_fail(LA_ERR_NO_MEMORY, who, "workspace allocation");
        }
        ws = own;
    }
    p.timeout = 1LL << 32;
    p.hold = -1;
    if (tiles_fit) tc_debug_take_timeout(&p.timeout, &p.hold);
    p.info = static_cast<int4 *>(ws);
    p.part = reinterpret_cast<float *>(p.info + blocks);
    e = cudaFuncSetAttribute(c.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, c.smem);
    if (e == cudaSuccess) {
        void *args[] = {&p, &maps[0], &maps[1]};  // the fp32 kernels take the first alone
        e = cudaLaunchKernel(c.kern, dim3((unsigned)blocks), dim3(kThreads), args, (size_t)c.smem, s);
        if (e == cudaSuccess) note_launches(1);
    }
    // The join is a dependent launch whose blocks start as the pieces' blocks end.  (Let in
    // from the start they cost 10 % of 1 x 131072 keys: 109 us, 98 us without.)
    if (e == cudaSuccess && blocks > 1) {
        const dim3 grid((unsigned)blocks - 1, (unsigned)p.row_tile);
        const unsigned threads = kJoin * ((unsigned)(d + 31) / 32 * 32);
        e = dtype == LA_F32
                ? tchost::launch_dependent(paged_join_kernel<float>, grid, threads, 0, s, p)
                : tchost::launch_dependent(paged_join_kernel<__nv_bfloat16>, grid, threads, 0, s, p);
        if (e == cudaSuccess) note_launches(1);
    }
    if (own) {
        const cudaError_t ef = cudaFreeAsync(own, s);
        if (e == cudaSuccess) e = ef;
    }
    return e == cudaSuccess ? LA_OK : layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
}

__attribute__((visibility("default")))
size_t la_decode_step_paged_workspace_bytes(int Hq, int Hk, int T, int d, la_dtype dtype) {
    if (Hk < 1 || Hq < 1 || Hq % Hk || T < 1 || d < 1 || d > LA_MAX_D) return 0;
    if (dtype != LA_F32 && dtype != LA_BF16) return 0;
    int sms = 0;
    if (tchost::sm_count(&sms) != cudaSuccess || sms <= 0) sms = 1;
    return workspace_of(blocks_of(sms), row_tile_of((long long)(Hq / Hk) * T, dtype), d);
}

}  // extern "C"

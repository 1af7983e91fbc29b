// New tokens into a paged cache (la_append_cache in include/linattn.h): keys and
// queries rotated by their position, keys and values to the pages that the table
// names,
//   p = lengths[b] + t,  cache[table[b][p / page_size]][h][p % page_size] = R(p) k_t,
//   (y1, y2) = (x1 cos a - x2 sin a, x2 cos a + x1 sin a),  a = (p + offset) f
// for each pair of features, angles as in la_qk_rope.cu.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "la_internal.h"
#include "la_layer.cuh"
#include "la_tc_host.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = LA_MAX_D / 2;
constexpr int kRows = 4;  // heads of a thread under way at a time

struct Tensor {
    const void *x;
    la_strides s;
};

struct Params {
    Tensor q, k, v;
    void *q_out, *k_cache, *v_cache;
    la_strides sq_out, sk_cache, sv_cache;
    const int *table, *lengths, *counts;
    long long table_stride, offset;
    int pages, page_size, max_pages;
    int B, Hq, Hk, T, d, half;
    // the split of the work, see append_kernel
    int lane_bits, token_bits;
    unsigned long long turns[kMaxPairs];
};

// cos and sin of a thread's V pairs, as the packed instructions take them.
template <int V, bool kInter>
struct Turn {
    float2 c[V], s[V];

    __device__ __forceinline__ void set(int i, float cs, float sn) {
        if (kInter || V == 1) {  // one pair: (x0, x1) (c, c) + (x1, x0) (-s, s)
            c[i] = make_float2(cs, cs);
            s[i] = make_float2(-sn, sn);
        } else {  // two pairs: x0 c - x1 s and x1 c + x0 s
            (i % 2 ? c[i / 2].y : c[i / 2].x) = cs;
            (i % 2 ? s[i / 2].y : s[i / 2].x) = sn;
        }
    }
    // e: V first and V second values, or V pairs
    __device__ __forceinline__ void apply(float (&e)[2 * V]) const {
        if (kInter || V == 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 x = make_float2(e[2 * i], e[2 * i + 1]);
                const float2 y =
                    __ffma2_rn(x, c[i], __fmul2_rn(make_float2(x.y, x.x), s[i]));
                e[2 * i] = y.x, e[2 * i + 1] = y.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 x0 = make_float2(e[2 * i], e[2 * i + 1]);
                const float2 x1 = make_float2(e[V + 2 * i], e[V + 2 * i + 1]);
                const float2 ns = make_float2(-s[i].x, -s[i].y);
                const float2 y0 = __ffma2_rn(x0, c[i], __fmul2_rn(x1, ns));
                const float2 y1 = __ffma2_rn(x1, c[i], __fmul2_rn(x0, s[i]));
                e[2 * i] = y0.x, e[2 * i + 1] = y0.y;
                e[V + 2 * i] = y1.x, e[V + 2 * i + 1] = y1.y;
            }
        }
    }
};

// A block takes 2^token_bits tokens, one for each part of its threads; the part's
// groups of 2^lane_bits threads take the token's heads (queries, keys, values) in turn.
// A thread keeps to two vectors of V features, the two halves of V pairs, in all heads,
// so that angles, position and page are found once for many of them, kRows of which are
// under way at a time.
//
// Bound by memory: 8 x 8192 tokens (fewer in some sequences) of 32 + 8 + 8 heads of 128
// bf16 values: 240 us, 6.2 TB/s.  (Two heads under way 272 us; three or four blocks per SM
// spill: 275 to 293 us.  Angles found for three heads at a time instead of twelve: 367 us.)
template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads, 2) append_kernel(const __grid_constant__ Params p) {
    const int unit = threadIdx.x & ((1 << p.lane_bits) - 1);
    const int group = threadIdx.x >> p.lane_bits;
    const int step = (kThreads >> p.lane_bits) >> p.token_bits;
    const long long token =
        ((long long)blockIdx.x << p.token_bits) + (group & ((1 << p.token_bits) - 1));
    if (token >= (long long)p.B * p.T) return;
    const int b = (int)(token / p.T), t = (int)(token - (long long)b * p.T);

    int at[2];
    if (kInter) {
        at[0] = 2 * V * unit;
        at[1] = at[0] + V;
    } else if (unit * V < p.half) {
        at[0] = unit * V;
        at[1] = at[0] + p.half;
    } else {
        at[0] = 2 * V * unit;  // 2 half + 2 (unit V - half)
        at[1] = at[0] + V;
    }
    if (at[0] >= p.d) return;
    const bool second = at[1] < p.d;

    const int before = p.lengths[b];
    const long long pos = (long long)before + t;
    // where its key and value go, if the cache has a place for them
    bool keep = before >= 0 && (!p.counts || t < p.counts[b]);
    long long page = 0, slot = 0;
    if (keep) {
        const long long column = pos / p.page_size;
        keep = column < p.max_pages;
        if (keep) {
            page = p.table[b * p.table_stride + column];
            slot = pos - column * p.page_size;
            keep = page >= 0 && page < p.pages;
        }
    }
    Turn<V, kInter> turn;
    bool all = true, any = false;  // of this thread's pairs are rotated
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int pair = unit * V + i;
        float c = 1.f, s = 0.f;
        if (pair < p.half) turn_of<sizeof(T) == 4>(pos + p.offset, p.turns[pair], &c, &s);
        all &= pair < p.half;
        any |= pair < p.half;
        turn.set(i, c, s);
    }

    // One side: this group's heads of H, `skip` heads of other sides having been dealt
    // out before.
    auto side = [&](const Tensor &in, void *out, const la_strides &so, long long to, int H,
                    int skip, bool rotate) {
        int h = (group >> p.token_bits) - skip % step;
        if (h < 0) h += step;
        const T *src = static_cast<const T *>(in.x) + b * in.s.b + t * in.s.n + h * in.s.h;
        T *dst = static_cast<T *>(out) + to + h * so.h;
        const long long src_step = step * in.s.h, dst_step = step * so.h;
        for (; h < H; h += kRows * step) {
            Pack<T, V> x[kRows][2];
#pragma unroll
            for (int i = 0; i < kRows; ++i, src += src_step)
                if (h + i * step < H) {
                    x[i][0] = *reinterpret_cast<const Pack<T, V> *>(src + at[0]);
                    if (second) x[i][1] = *reinterpret_cast<const Pack<T, V> *>(src + at[1]);
                }
#pragma unroll
            for (int i = 0; i < kRows; ++i, dst += dst_step) {
                if (h + i * step >= H) continue;
                // values, and features beyond the rotated ones, pass bit for bit
                if (rotate && any) {
                    float e[2 * V];
                    widen(&x[i][0], e);
                    if (second) widen(&x[i][1], e + V);
                    turn.apply(e);
                    Pack<T, V> y[2];
                    narrow<T, V>(y[0].v, e);
                    narrow<T, V>(y[1].v, e + V);
                    if (kInter && !all)  // neighbouring pairs of which some pass
#pragma unroll
                        for (int j = 0; j < 2 * V; ++j)
                            if (unit * V + j / 2 >= p.half) y[j / V].v[j % V] = x[i][j / V].v[j % V];
                    *reinterpret_cast<Pack<T, V> *>(dst + at[0]) = y[0];
                    if (second) *reinterpret_cast<Pack<T, V> *>(dst + at[1]) = y[1];
                } else {
                    *reinterpret_cast<Pack<T, V> *>(dst + at[0]) = x[i][0];
                    if (second) *reinterpret_cast<Pack<T, V> *>(dst + at[1]) = x[i][1];
                }
            }
        }
    };
    side(p.q, p.q_out, p.sq_out, b * p.sq_out.b + t * p.sq_out.n, p.Hq, 0, true);
    if (!keep) return;
    side(p.k, p.k_cache, p.sk_cache, page * p.sk_cache.b + slot * p.sk_cache.n, p.Hk, p.Hq, true);
    side(p.v, p.v_cache, p.sv_cache, page * p.sv_cache.b + slot * p.sv_cache.n, p.Hk,
         p.Hq + p.Hk, false);
}

template <typename T>
la_status launch(const char *who, Params &p, int interleaved, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = tchost::sm_count(&sms);
    if (e != cudaSuccess) return layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    // values per access: the most at which every row of every tensor is aligned
    unsigned long long all = (unsigned)((interleaved ? 2 * p.half : p.half) | p.d |
                                        16 / (int)sizeof(T));
    auto add = [&](const void *x, const la_strides &s, int n0, int n1, int n2) {
        if (n1 == 0) return;
        all |= (uintptr_t)x / sizeof(T);
        if (n0 > 1) all |= (unsigned long long)s.b;
        if (n1 > 1) all |= (unsigned long long)s.h;
        if (n2 > 1) all |= (unsigned long long)s.n;
    };
    add(p.q.x, p.q.s, p.B, p.Hq, p.T);
    add(p.q_out, p.sq_out, p.B, p.Hq, p.T);
    add(p.k.x, p.k.s, p.B, p.Hk, p.T);
    add(p.v.x, p.v.s, p.B, p.Hk, p.T);
    add(p.k_cache, p.sk_cache, p.pages, p.Hk, p.page_size);
    add(p.v_cache, p.sv_cache, p.pages, p.Hk, p.page_size);
    const int v = (int)(all & (0 - all));
    const int units = (p.d + 2 * v - 1) / (2 * v);
    while (1 << p.lane_bits < units) ++p.lane_bits;
    // More tokens per block while a thread has fewer than 12 heads of its token, whose
    // angles serve them all, and enough blocks are left for every SM.
    const int groups = kThreads >> p.lane_bits, rows = p.Hq + 2 * p.Hk;
    const long long tokens = (long long)p.B * p.T;
    while ((2 << p.token_bits) <= groups && rows * (1 << p.token_bits) < 12 * groups &&
           tokens >> (p.token_bits + 1) >= 6 * sms)
        ++p.token_bits;
    const long long blocks = (tokens + (1 << p.token_bits) - 1) >> p.token_bits;
    if (blocks > 0x7fffffff) return layer_fail(LA_ERR_UNSUPPORTED, who, "problem too large");
    auto go = [&](auto kern) {
        kern<<<(unsigned)blocks, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    };
    constexpr int kMost = 16 / (int)sizeof(T);
    if (v == kMost)
        e = interleaved ? go(append_kernel<T, kMost, true>) : go(append_kernel<T, kMost, false>);
    else if (v == 4)
        e = interleaved ? go(append_kernel<T, 4, true>) : go(append_kernel<T, 4, false>);
    else if (v == 2)
        e = interleaved ? go(append_kernel<T, 2, true>) : go(append_kernel<T, 2, false>);
    else
        e = interleaved ? go(append_kernel<T, 1, true>) : go(append_kernel<T, 1, false>);
    if (e != cudaSuccess) return layer_fail(LA_ERR_CUDA, who, cudaGetErrorString(e));
    note_launches(1);
    return LA_OK;
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

__attribute__((visibility("default")))
la_status la_append_cache(const void *q, const void *k, const void *v, void *q_out,
                          const la_cache *cache, const int *counts, const la_strides *strides,
                          const la_rope *rope, int B, int Hq, int Hk, int T, int d,
                          la_dtype dtype, la_stream_t stream) {
    const char *who = "la_append_cache";
    if (Hq < 0 || T < 0) return layer_fail(LA_ERR_INVALID_ARG, who, "negative Hq or T");
    la_status st = check_cache(who, cache, B, Hk, d, dtype);
    if (st != LA_OK) return st;
    // a thread's heads are counted in 32 bits, up to kRows kThreads behind the last one
    if (Hq + 2LL * Hk >= 0x7fffffff - 4 * kRows * kThreads)
        return layer_fail(LA_ERR_UNSUPPORTED, who, "too many heads");
    Params p{};
    if (rope && rope->rotary_dim != 0) {
        const int R = rope->rotary_dim;
        if (R < 0 || R > d || R % 2)
            return layer_fail(LA_ERR_INVALID_ARG, who, "rotary_dim must be even and in 0..d");
        if (rope->interleaved != 0 && rope->interleaved != 1)
            return layer_fail(LA_ERR_INVALID_ARG, who, "interleaved must be 0 or 1");
        if (!rope->frequencies) return layer_fail(LA_ERR_INVALID_ARG, who, "null frequencies");
        if (rope->positions)
            return layer_fail(LA_ERR_INVALID_ARG, who, "positions are those in the cache");
        for (int i = 0; i < R / 2; ++i) {
            if (!(std::fabs(rope->frequencies[i]) <= 1e9))  // also rejects NaN
                return layer_fail(LA_ERR_INVALID_ARG, who,
                                  "frequencies must lie in [-1e9, 1e9]");
            p.turns[i] = turns_of(rope->frequencies[i]);
        }
        p.half = R / 2;
        p.offset = rope->offset;
    }
    if (B == 0 || T == 0 || Hq + Hk == 0) return LA_OK;
    const uintptr_t elem = dtype == LA_F32 ? 4 : 2;
    const void *in[3] = {q, k, v};
    Tensor *to[3] = {&p.q, &p.k, &p.v};
    for (int i = 0; i < 3; ++i) {
        const int H = i ? Hk : Hq;
        if (H == 0) continue;
        *to[i] = {in[i], strides ? strides[i] : contiguous(H, T, d)};
        if (!in[i]) return layer_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
        if ((uintptr_t)in[i] % elem)
            return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
        if (negative(to[i]->s)) return layer_fail(LA_ERR_INVALID_ARG, who, "negative stride");
    }
    if (Hq) {
        p.q_out = q_out;
        p.sq_out = strides ? strides[3] : contiguous(Hq, T, d);
        if (!q_out) return layer_fail(LA_ERR_INVALID_ARG, who, "null tensor pointer");
        if ((uintptr_t)q_out % elem)
            return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned tensor pointer");
        if (negative(p.sq_out)) return layer_fail(LA_ERR_INVALID_ARG, who, "negative stride");
        if (!rows_disjoint(p.sq_out, B, Hq, T, d))
            return layer_fail(LA_ERR_INVALID_ARG, who, "output rows overlap");
        if (q_out == q && (p.sq_out.b != p.q.s.b || p.sq_out.h != p.q.s.h || p.sq_out.n != p.q.s.n))
            return layer_fail(LA_ERR_INVALID_ARG, who, "in place needs equal strides");
        if (Hk && (q_out == k || q_out == v || q_out == cache->k || q_out == cache->v))
            return layer_fail(LA_ERR_INVALID_ARG, who, "q_out aliases another tensor");
    }
    if (Hk) {
        for (const void *x : in)
            if (x && (x == cache->k || x == cache->v))
                return layer_fail(LA_ERR_INVALID_ARG, who, "the cache aliases another tensor");
        if (!rows_disjoint(cache->k_strides, cache->pages, Hk, cache->page_size, d) ||
            !rows_disjoint(cache->v_strides, cache->pages, Hk, cache->page_size, d))
            return layer_fail(LA_ERR_INVALID_ARG, who, "cache rows overlap");
        p.k_cache = cache->k;
        p.v_cache = cache->v;
        p.sk_cache = cache->k_strides;
        p.sv_cache = cache->v_strides;
        if (cache->pages == 0) p.k_cache = p.v_cache = nullptr;  // no token has a place
    }
    if ((uintptr_t)counts % 4) return layer_fail(LA_ERR_INVALID_ARG, who, "unaligned counts");
    p.table = cache->table;
    p.lengths = cache->lengths;
    p.counts = counts;
    p.table_stride = cache->table_stride;
    p.pages = cache->pages;
    p.page_size = cache->page_size;
    p.max_pages = cache->max_pages;
    p.B = B;
    p.Hq = Hq;
    p.Hk = Hk;
    p.T = T;
    p.d = d;
    const int interleaved = rope && rope->rotary_dim ? rope->interleaved : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == LA_F32 ? launch<float>(who, p, interleaved, s)
                           : launch<__nv_bfloat16>(who, p, interleaved, s);
}

}  // extern "C"

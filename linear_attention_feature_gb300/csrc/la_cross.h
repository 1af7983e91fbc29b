// Linear cross attention: what its translation units share (la_forward_cross,
// la_backward_cross, la_decode_step_cross in include/linattn.h).
#pragma once

#include <cmath>

#include "la_internal.h"

namespace la {
namespace cross {

struct Shape {
    int B, Hq, Hk, N, M, d;
    int phi, norm;       // elu(x) + 1, else the identity; with the denominator
    const int *lengths;  // [B] tokens on the keys' side, or NULL: M
    int G() const { return Hq / Hk; }
    long long heads() const { return (long long)B * Hk; }  // states
    long long state() const { return (long long)d * d; }
};

// A [B][H][L][d] tensor, read or written.
struct Rows {
    void *x;
    la_strides s;
};

// Tokens of one head whose sums make up a state, cut into `segs` parts of `per`.
struct Cut {
    int segs, tile;  // tile: the side of a block's sums in fp32
    long long per;
};

// The tensor-core kernels (la_cross_tc.cu): whether they take these bf16 tensors (the
// queries' side and the keys'), their workspace and their launches.  `dependent`: S and z
// come from the kernel before on the stream, which lets this one start early.
bool tc_rows(const Shape &sh, const Rows *q_side, int nq, const Rows *k_side, int nk,
             const float *S, const float *z);
size_t tc_workspace(const Shape &sh, int sms, bool backward);
cudaError_t tc_state(const Shape &sh, Rows k, Rows v, float *S, float *z, char *ws, int sms,
                     int *status, cudaStream_t s);
cudaError_t tc_read(const Shape &sh, Rows q, Rows out, const float *S, const float *z,
                    bool dependent, int sms, int *status, cudaStream_t s);
cudaError_t tc_backward(const Shape &sh, Rows dout, Rows q, Rows k, Rows v, const float *S,
                        const float *z, Rows dq, Rows dk, Rows dv, char *ws, int sms, int *status,
                        cudaStream_t s);

#ifdef __CUDACC__
__device__ __forceinline__ int tokens_of(const int *lengths, int b, int M) {
    return lengths ? min(max(lengths[b], 0), M) : M;
}
// r and t of a row whose denominator is 0, which adds nothing to dS and dz whatever its dy
// is: t is not infinite where r = 0 is 1 / den.
__device__ __forceinline__ float2 no_row() { return make_float2(0.f, INFINITY); }
__device__ __forceinline__ bool is_none(float2 rt) { return rt.x == 0.f && rt.y == INFINITY; }
#endif

// ---- The parts of a call without those tiles: fp32 in la_cross.cu, bf16 in
// la_cross_half.cu.

// Sums of outer products.
struct SumParams {
    const void *x, *y;  // rows of features (phi is taken) and of values
    la_strides sx, sy;
    const float2 *rt;    // backward: r and t of each row of x, [B][Hk][group][L], or no_row()
    const int *lengths;  // forward, or NULL
    int Hk, group, L, d, phi, segs;
    long long per, heads;
    float *S, *z;  // [segs][heads][d d], [segs][heads][d]
};

// Rows times a state.
struct ReadParams {
    const void *x;
    void *y;
    la_strides sx, sy;
    const float *S, *z;
    const int *lengths;  // rows behind are written as 0, or NULL
    int Hk, group, L, d, phi, norm;
};

struct GradParams {
    const void *y, *x;  // what is multiplied, and what phi is taken of
    void *dx;
    la_strides sy, sx, sdx;
    const float *S, *z;
    float2 *rt;          // q's side: written
    const int *lengths;  // k's side: rows behind are written as 0, or NULL
    int Hk, group, L, d, phi, norm, keys;
};

// `heads`: of the rows' tensor, of all sequences.
cudaError_t half_sums(const SumParams &p, cudaStream_t s);
cudaError_t half_read(const ReadParams &p, long long heads, cudaStream_t s);
cudaError_t half_grads(const GradParams &p, long long heads, cudaStream_t s);

}  // namespace cross
}  // namespace la

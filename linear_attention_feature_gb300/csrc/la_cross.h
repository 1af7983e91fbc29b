// Linear cross attention: what its translation units share (la_forward_cross,
// la_backward_cross, la_decode_step_cross in include/linattn.h).
#pragma once

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
    int segs;
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

}  // namespace cross
}  // namespace la

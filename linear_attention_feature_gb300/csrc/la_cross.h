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

}  // namespace cross
}  // namespace la

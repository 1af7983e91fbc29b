// The backward scan of la_backward_recurrence: a translation unit of its own,
// so that the two directions compile side by side.
#include "la_recurrence.cuh"

namespace la {
namespace rec {

la_status launch_backward(const char *who, Params &p, la_gate gate, la_dtype dtype,
                          la_dtype gate_dtype, Workspace ws, cudaStream_t s) {
    return launch<true>(who, p, gate, dtype, gate_dtype, ws, s);
}

}  // namespace rec
}  // namespace la

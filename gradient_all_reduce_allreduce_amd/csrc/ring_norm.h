// Arguments of the all-reduce that leaves its result's sum of squares
// (ring_norm.hip): the ring's, then its own.
#pragma once

#include "ring_reduce_impl.h"

namespace ddp {
namespace rr {

struct RingNormArgs {
    RingArgs ring;
    double* partials;    // one sum of squares per workgroup of this launch
    int32_t one_copy;    // write the result to rank 0 only
};

}  // namespace rr

const void* ring_norm_kernel(int P, bool in_bf16, bool out_bf16, int scalar);

}  // namespace ddp

// Arguments of the all-reduce that leaves its result's sum of squares
// (ring_norm.hip): the ring's, then its own.
#pragma once

#include "ring_reduce_impl.h"

namespace ddp {
namespace rr {

struct RingNormArgs {
    RingArgs ring;
    double* partials;    // one sum of squares per workgroup of this launch
    uint64_t* zero;      // cleared by this launch's first workgroup, or null
    int32_t one_copy;    // write the result to rank 0 only
};

}  // namespace rr

// Resident one-wave workgroups per CU by element types (f32 -> f32, f32 ->
// bf16, bf16 -> f32, bf16 -> bf16) and rank count P = 1..16 (index 0 unused;
// P = 9, 11, 13 and 15 interpolate), the fastest of 2..32 and no cap on
// 200M elements of all ranks together.  With every rank written the best is
// the plain all-reduce's or one or two more: a workgroup lives a little longer
// for its sum.  With one copy most of the traffic is reads, and more of them
// want to be in flight: 48-96 KiB per CU.
constexpr signed char kRingNormWg[4][17] = {
    //   P: 1   2   3   4   5   6  7  8  9 10 11 12 13 14 15 16
    {0, 10, 5, 10, 8, 8, 6, 5, 5, 5, 5, 5, 4, 4, 4, 4, 4},
    {0, 14, 10, 16, 12, 10, 8, 8, 6, 7, 8, 7, 6, 6, 6, 5, 5},
    {0, 14, 10, 16, 12, 10, 8, 8, 6, 7, 8, 7, 6, 6, 6, 5, 5},
    {0, 10, 10, 14, 10, 10, 8, 6, 6, 6, 6, 6, 5, 5, 5, 5, 4},
};
constexpr signed char kRingNormOneWg[4][17] = {
    //   P: 1   2   3   4   5   6   7   8   9 10 11 12 13 14 15 16
    {0, 10, 6, 16, 12, 12, 10, 10, 8, 8, 8, 7, 6, 6, 6, 5, 5},
    {0, 14, 12, 20, 14, 16, 14, 12, 10, 9, 8, 8, 8, 8, 8, 7, 6},
    {0, 14, 20, 24, 24, 32, 24, 20, 16, 16, 16, 16, 16, 14, 12, 11, 10},
    {0, 10, 16, 24, 24, 20, 16, 14, 12, 12, 12, 11, 10, 10, 10, 9, 8},
};
constexpr int ring_norm_wg_per_cu(int P, bool in_bf16, bool out_bf16, bool one_copy) {
    return (one_copy ? kRingNormOneWg : kRingNormWg)[(in_bf16 ? 2 : 0) + (out_bf16 ? 1 : 0)][P];
}

const void* ring_norm_kernel(int P, bool in_bf16, bool out_bf16, int scalar);

}  // namespace ddp

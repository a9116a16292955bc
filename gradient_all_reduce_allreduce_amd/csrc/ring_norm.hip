// ring_norm.hip -- the ring all-reduce that also leaves the sum of squares of
// its result, for gfx950: the ring's tile code (ring_reduce_impl.h) with the
// squares taken on the way.
//
// The global norm of the reduced gradient needs every element once more;
// here its square is taken from the registers the result is stored from (as
// it is written: rounded for bf16), in float64, where it is exact.  Each
// workgroup -- one wave, one tile -- adds its lanes in a fixed order and
// writes one partial; a second, small launch adds the partials
// (grad_norm.hip).  The squares and the wave's sum cost nothing that shows: at
// P = 8, 25.6M float32, all ranks written, 251 us without the second launch
// against 248 for the plain all-reduce, and 257 (6.4 TB/s) with it.  86.6M bf16
// into one float32 copy 268 us, 6.5 TB/s (the plain call writes 8 copies).
#include "grad_vec.h"
#include "ring_norm.h"

namespace ddp {
namespace rr {
namespace {

typedef const __attribute__((address_space(4))) RingNormArgs* KRingNorm;

__device__ __forceinline__ KRingNorm norm_args() {
    return (KRingNorm)(__builtin_amdgcn_kernarg_segment_ptr());
}

// Leaves the wave's sum.  The first workgroup of a launch also clears the count
// that the partials' sum starts from (grad_norm.hip).
__device__ __forceinline__ void leave(KRingNorm a, double sq) {
    sq = gv::wave_sum63(sq);
    if (threadIdx.x == 63) {
        a->partials[blockIdx.x] = sq;
        if (blockIdx.x == 0 && a->zero != nullptr) *a->zero = 0;
    }
}

template <int P, bool INB, bool OUTB>
__global__ __launch_bounds__(kBlock) void ring_norm_kernel(RingNormArgs) {
    const KRingNorm a = norm_args();
    double sq = 0.0;
    ring_reduce_body<P, INB, OUTB, false, true>(&sq, a->one_copy != 0);
    leave(a, sq);
}

template <int P, bool INB, bool OUTB>
__global__ __launch_bounds__(kBlock) void ring_norm_scalar_kernel(RingNormArgs) {
    const KRingNorm a = norm_args();
    const uint32_t i = blockIdx.x * kBlock + threadIdx.x;
    double sq = 0.0;
    if (i < a->ring.n) process_element<P, INB, OUTB, false, true>(&a->ring, i, &sq, a->one_copy != 0);
    leave(a, sq);
}

template <bool INB, bool OUTB, bool SCALAR>
const void* ring_norm_kernel_for(int P) {
    switch (P) {
#define DDP_CASE(p)                                                                                \
    case p:                                                                                        \
        return SCALAR ? reinterpret_cast<const void*>(&ring_norm_scalar_kernel<p, INB, OUTB>)      \
                      : reinterpret_cast<const void*>(&ring_norm_kernel<p, INB, OUTB>);
        DDP_CASE(1) DDP_CASE(2) DDP_CASE(3) DDP_CASE(4)
        DDP_CASE(5) DDP_CASE(6) DDP_CASE(7) DDP_CASE(8)
        DDP_CASE(9) DDP_CASE(10) DDP_CASE(11) DDP_CASE(12)
        DDP_CASE(13) DDP_CASE(14) DDP_CASE(15) DDP_CASE(16)
#undef DDP_CASE
        default:
            return nullptr;
    }
}

}  // namespace
}  // namespace rr

const void* ring_norm_kernel(int P, bool in_bf16, bool out_bf16, int scalar) {
    if (in_bf16) {
        if (out_bf16) return scalar ? rr::ring_norm_kernel_for<true, true, true>(P) : rr::ring_norm_kernel_for<true, true, false>(P);
        return scalar ? rr::ring_norm_kernel_for<true, false, true>(P) : rr::ring_norm_kernel_for<true, false, false>(P);
    }
    if (out_bf16) return scalar ? rr::ring_norm_kernel_for<false, true, true>(P) : rr::ring_norm_kernel_for<false, true, false>(P);
    return scalar ? rr::ring_norm_kernel_for<false, false, true>(P) : rr::ring_norm_kernel_for<false, false, false>(P);
}

}  // namespace ddp

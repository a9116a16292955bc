// mx4_reduce.hip -- the all-reduce of rank gradients in microscaled 4-bit
// floating point, for gfx950.
//
// Per element, float32, one rounding per operation:
//     g = q_0 + q_1 + ... + q_{P-1}            the ranks' values in rank order
//     g = g / P                                 Mean
// written as float32 or bf16 to one copy or to every rank, or coded again (as
// mx4.hip does, with a left-over of the owner's) for the way back.  The codes
// of a block travel once and whole, to an owner that adds the P copies, so the
// order is the same for every element, whatever the chunks.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch_mx.h"
#include "mx.h"

namespace ddp {
namespace {

struct ReduceArgs {
    const char* codes[kMaxRanks];
    const char* scales[kMaxRanks];
    char* out[kMaxRanks];
    char* out_scales[kMaxRanks];
    char* left;
    double* partials;
    uint64_t* zero;
    int64_t n;
    uint32_t tiles;
    int32_t n_out;
    int32_t mean;
    int32_t left_type;
};
typedef const __attribute__((address_space(4))) ReduceArgs* KReduce;

template <bool BF16>
__device__ __forceinline__ void add_left(float (&g)[8], const char* left, int64_t i, int64_t n, bool whole) {
    const mx::Oct<BF16> r = mx::load_oct<BF16>(left, i, n, whole);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] += mx::oct_elem<BF16>(r, e);
}

// OUT: 0 float32, 1 bf16, 2 coded.
template <int P, int OUT>
__global__ __launch_bounds__(mx::kWave) void mx4_reduce_kernel(ReduceArgs) {
    const KReduce a = (KReduce)(__builtin_amdgcn_kernarg_segment_ptr());
    const int64_t n = a->n;
    const uint32_t tiles = a->tiles;
    double sq = 0.0;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t at = tile * kMxTileElems;
        const int64_t i = at + threadIdx.x * 8;
        const bool whole = at + kMxTileElems <= n || i + 8 <= n;
        const bool held = i / DDP_MX_BLOCK * DDP_MX_BLOCK < n;     // in a block of the row
        uint32_t c[P], s[P];
#pragma unroll
        for (int r = 0; r < P; ++r) {
            c[r] = held ? mx::load_codes(a->codes[r], i) : 0u;
            s[r] = held ? mx::load_scale(a->scales[r], i) : 0u;
        }
        float g[8];
        mx::decode8(c[0], mx::scale_of(s[0]), g);
#pragma unroll
        for (int r = 1; r < P; ++r) {
            float x[8];
            mx::decode8(c[r], mx::scale_of(s[r]), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] += x[e];
        }
        if (a->mean) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = rr::mean_of<P>(g[e]);
        }
        if constexpr (OUT == 2) {
            if (a->left_type == 1) add_left<false>(g, a->left, i, n, whole);
            if (a->left_type == 2) add_left<true>(g, a->left, i, n, whole);
            // behind the row's end the codes are zero
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = i + e < n ? g[e] : 0.0f;
            const mx::Coded q = mx::quantize8(g);
            float x[8];
            mx::decode8(q.codes, mx::scale_of(q.scale), x);
            if (held) {
                for (int r = 0; r < a->n_out; ++r) {
                    mx::store_codes(a->out[r], i, q.codes);
                    if ((threadIdx.x & 3) == 0) mx::store_scale(a->out_scales[r], i, q.scale);
                }
            }
            if (a->left_type != 0 && q.finite) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = g[e] - x[e];
                if (a->left_type == 1) mx::store_oct<false>(a->left, i, n, whole, mx::pack_oct<false>(y));
                if (a->left_type == 2) mx::store_oct<true>(a->left, i, n, whole, mx::pack_oct<true>(y));
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = x[e];
        } else {
            const mx::Oct<OUT == 1> o = mx::pack_oct<OUT == 1>(g);
            for (int r = 0; r < a->n_out; ++r) mx::store_oct<OUT == 1>(a->out[r], i, n, whole, o);
        }
        if (a->partials != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e < n) sq = rr::square_to(sq, rr::written<OUT == 1>(g[e]));
        }
    }
    if (a->partials != nullptr) {
        sq = gv::wave_sum63(sq);
        if (threadIdx.x == 63) {
            a->partials[blockIdx.x] = sq;
            if (blockIdx.x == 0 && a->zero != nullptr) *a->zero = 0;
        }
    }
}

template <int OUT>
const void* kernel_for(int P) {
    switch (P) {
#define DDP_CASE(p) \
    case p:         \
        return reinterpret_cast<const void*>(&mx4_reduce_kernel<p, OUT>);
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

int64_t mx4_reduce_workgroups(int64_t n) { return std::min<int64_t>(mx_tiles(n), kMaxWaveGrid); }

int launch_mx4_reduce(const Mx4Reduce& l, const char** msg) {
    ReduceArgs a{};
    for (int r = 0; r < l.P; ++r) {
        a.codes[r] = static_cast<const char*>(l.codes[r]);
        a.scales[r] = static_cast<const char*>(l.scales[r]);
    }
    for (int r = 0; r < l.n_out; ++r) {
        a.out[r] = static_cast<char*>(l.out[r]);
        a.out_scales[r] = static_cast<char*>(l.out_scales[r]);
    }
    a.left = static_cast<char*>(l.left);
    a.partials = l.partials;
    a.zero = l.zero;
    a.n = l.n;
    a.tiles = static_cast<uint32_t>(mx_tiles(l.n));
    a.n_out = l.n_out;
    a.mean = l.mean;
    a.left_type = l.left_type;
    const void* fn = l.out_type == 0 ? kernel_for<0>(l.P) : l.out_type == 1 ? kernel_for<1>(l.P) : kernel_for<2>(l.P);
    void* args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3(static_cast<unsigned>(mx4_reduce_workgroups(l.n))), dim3(mx::kWave),
                                         args, 0, static_cast<hipStream_t>(l.stream));
    if (e == hipSuccess) return 0;
    *msg = "hipLaunchKernel(mx4_reduce)";
    return static_cast<int>(e);
}

}  // namespace ddp

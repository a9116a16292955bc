// mx4.hip -- gradients to microscaled 4-bit floating point and back, for
// gfx950.
//
// Quantise, for every block of 32 elements of a rank's row:
//     t = gradient + left-over                 float32, one rounding
//     s = the smallest power of two that lets no element round past 6 s
//     code = the nearest level of t / s, ties to even;   q = its value
//     left-over = t - q                        exact in float32
// (no left-over: t is the gradient).  The rounding error of one step goes into
// the next one's gradient, so that what is sent adds up to what was computed.
// A block that holds an infinity or a NaN is sent as NaN and its left-over
// stays as it was.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch_mx.h"
#include "mx.h"

namespace ddp {
namespace {

struct Mx4Args {
    char* values[kMaxRanks];
    char* left[kMaxRanks];
    char* codes[kMaxRanks];
    char* scales[kMaxRanks];
    int64_t n;
    uint32_t tiles;
};
typedef const __attribute__((address_space(4))) Mx4Args* KMx4;

// LEFT: the left-over, 0 none, 1 float32, 2 bf16.
template <bool BF16, int LEFT>
__global__ __launch_bounds__(mx::kWave) void mx4_quantize_kernel(Mx4Args) {
    const KMx4 a = (KMx4)(__builtin_amdgcn_kernarg_segment_ptr());
    const char* const in = a->values[blockIdx.y];
    char* const left = a->left[blockIdx.y];
    char* const codes = a->codes[blockIdx.y];
    char* const scales = a->scales[blockIdx.y];
    const int64_t n = a->n;
    const uint32_t tiles = a->tiles;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t at = tile * kMxTileElems;
        const int64_t i = at + threadIdx.x * 8;
        const bool whole = at + kMxTileElems <= n || i + 8 <= n;
        const mx::Oct<BF16> g = mx::load_oct<BF16>(in, i, n, whole);
        float t[8];
        mx::Oct<LEFT == 2> r;
        if constexpr (LEFT != 0) r = mx::load_oct<LEFT == 2>(left, i, n, whole);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t[e] = mx::oct_elem<BF16>(g, e);
            if constexpr (LEFT != 0) t[e] += mx::oct_elem<LEFT == 2>(r, e);
        }
        const mx::Coded q = mx::quantize8(t);
        if (i / DDP_MX_BLOCK * DDP_MX_BLOCK < n) {
            mx::store_codes(codes, i, q.codes);
            if ((threadIdx.x & 3) == 0) mx::store_scale(scales, i, q.scale);
        }
        if constexpr (LEFT != 0) {
            if (q.finite) {
                float x[8];
                mx::decode8(q.codes, mx::scale_of(q.scale), x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = t[e] - x[e];
                mx::store_oct<LEFT == 2>(left, i, n, whole, mx::pack_oct<LEFT == 2>(x));
            }
        }
    }
}

template <bool BF16>
__global__ __launch_bounds__(mx::kWave) void mx4_dequantize_kernel(Mx4Args) {
    const KMx4 a = (KMx4)(__builtin_amdgcn_kernarg_segment_ptr());
    char* const out = a->values[blockIdx.y];
    const char* const codes = a->codes[blockIdx.y];
    const char* const scales = a->scales[blockIdx.y];
    const int64_t n = a->n;
    const uint32_t tiles = a->tiles;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t at = tile * kMxTileElems;
        const int64_t i = at + threadIdx.x * 8;
        if (i >= n) continue;
        float x[8];
        mx::decode8(mx::load_codes(codes, i), mx::scale_of(mx::load_scale(scales, i)), x);
        mx::store_oct<BF16>(out, i, n, at + kMxTileElems <= n || i + 8 <= n, mx::pack_oct<BF16>(x));
    }
}

int launch(const void* fn, const Mx4Launch& l, int wg_per_cu, const char* what, const char** msg) {
    if (l.n == 0) return 0;
    Mx4Args a{};
    for (int r = 0; r < l.P; ++r) {
        a.values[r] = static_cast<char*>(const_cast<void*>(l.values[r]));
        a.left[r] = static_cast<char*>(l.left[r]);
        a.codes[r] = static_cast<char*>(l.codes[r]);
        a.scales[r] = static_cast<char*>(l.scales[r]);
    }
    a.n = l.n;
    a.tiles = static_cast<uint32_t>(mx_tiles(l.n));
    // a grid holds fewer than 2^32 lanes
    const unsigned grid = std::min(a.tiles, kMaxWaveGrid / static_cast<unsigned>(l.P));
    void* args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3(grid, static_cast<unsigned>(l.P)), dim3(mx::kWave), args,
                                         lds_reserve(wg_per_cu), static_cast<hipStream_t>(l.stream));
    if (e == hipSuccess) return 0;
    *msg = what;
    return static_cast<int>(e);
}

}  // namespace

int launch_mx4_quantize(const Mx4Launch& l, const char** msg) {
    const void* const fns[2][3] = {
        {reinterpret_cast<const void*>(&mx4_quantize_kernel<false, 0>),
         reinterpret_cast<const void*>(&mx4_quantize_kernel<false, 1>),
         reinterpret_cast<const void*>(&mx4_quantize_kernel<false, 2>)},
        {reinterpret_cast<const void*>(&mx4_quantize_kernel<true, 0>),
         reinterpret_cast<const void*>(&mx4_quantize_kernel<true, 1>),
         reinterpret_cast<const void*>(&mx4_quantize_kernel<true, 2>)}};
    return launch(fns[l.bf16][l.left_type], l, 0, "hipLaunchKernel(mx4_quantize)", msg);
}

int launch_mx4_dequantize(const Mx4Launch& l, const char** msg) {
    const void* const fns[2] = {reinterpret_cast<const void*>(&mx4_dequantize_kernel<false>),
                                reinterpret_cast<const void*>(&mx4_dequantize_kernel<true>)};
    return launch(fns[l.bf16], l, 0, "hipLaunchKernel(mx4_dequantize)", msg);
}

}  // namespace ddp

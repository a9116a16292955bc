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
//
// Bound by HBM: gradient and left-over in, left-over and 17/32 byte out, against
// some 10 instructions an element.  8 ranks of 25.6M: bf16 with bf16 left-over
// 206 us, 6.5 TB/s; float32 with float32 398 us, 6.4; bf16 alone 84 us, 6.2.  One
// rank of 252M bf16 with float32 left-over 414 us, 6.4; from 12 bytes into a line
// on, so that every access straddles lines, 443.  Back to bf16 80 us, 6.5 TB/s, to
// float32 147, 6.3.
//
// Layout (mx.h): a wave takes 2 spans of 512 elements, all loads first.  One span
// leaves too little in flight (bf16 alone 92 us) and starts nearly as many waves
// as the dispatcher can; with 4 a float32 row's waves hold too much (439 us
// instead of 398).  Short rows are quantised with one: 8 bf16 rows of 1,000
// elements with bf16 left-overs 3.8 us instead of 5.1, of 262,144 4.3 and 4.4, of
// 4.2M 39.6 and 37.5 (reading back: no difference).  A workgroup's 4,096 elements have 128 bytes of scales: one
// line, written by one CU.  By workgroups per CU 0 (full), 2, 3, 4, 5, 6, 8: bf16
// with left-over 212 236 225 206 207 212 211 us, float32 without 152 180 158 151
// 145 146 148, bf16 without 86 132 109 95 89 85 85.
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
constexpr bool kWide = !BF16 || LEFT == 1;

template <bool BF16, int LEFT, bool WHOLE>
__device__ __forceinline__ void quantize_span(const mx::Raw& g, const mx::Raw& r, char* left, char* codes, char* scales,
                                              int64_t at, int64_t n) {
    constexpr bool W = kWide<BF16, LEFT>;
    float t[8];
    mx::values_of<BF16, W>(g, t);
    if constexpr (LEFT != 0) {
        float x[8];
        mx::values_of<LEFT == 2, W>(r, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] += x[e];
    }
    const mx::Coded q = mx::quantize8<W>(t);
    mx::store_coded<W, WHOLE>(codes, scales, at, n, mx::shared_codes<W>(q.codes), q.scales);
    if constexpr (LEFT != 0) {
        float x[8];
        mx::decode8(q.codes, q.scales, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = t[e] - x[e];
        mx::store_values<LEFT == 2, W, WHOLE>(left, at, n, x, q.finite_a, q.finite_b);
    }
}

template <bool BF16, int LEFT, int U>
__global__ __launch_bounds__(kMxLanes) void mx4_quantize_kernel(Mx4Args) {
    constexpr bool W = kWide<BF16, LEFT>;
    const KMx4 a = (KMx4)(__builtin_amdgcn_kernarg_segment_ptr());
    const char* const in = a->values[blockIdx.y];
    char* const left = a->left[blockIdx.y];
    char* const codes = a->codes[blockIdx.y];
    char* const scales = a->scales[blockIdx.y];
    const int64_t n = a->n;
    const uint32_t tiles = a->tiles;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t at = mx::wave_start<U>(tile);
        mx::Raw g[U], r[U];
        if (at + U * mx::kMxSpan <= n) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                g[u] = mx::load_raw<BF16, W, true>(in, at + u * mx::kMxSpan, n);
                if constexpr (LEFT != 0) r[u] = mx::load_raw<LEFT == 2, W, true>(left, at + u * mx::kMxSpan, n);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                quantize_span<BF16, LEFT, true>(g[u], r[u], left, codes, scales, at + u * mx::kMxSpan, n);
        } else {
            for (int64_t i = at; i < n; i += mx::kMxSpan) {
                g[0] = mx::load_raw<BF16, W, false>(in, i, n);
                if constexpr (LEFT != 0) r[0] = mx::load_raw<LEFT == 2, W, false>(left, i, n);
                quantize_span<BF16, LEFT, false>(g[0], r[0], left, codes, scales, i, n);
            }
        }
    }
}

template <bool BF16, bool WHOLE>
__device__ __forceinline__ void dequantize_span(uint32_t c, uint32_t s, char* out, int64_t at, int64_t n,
                                                mx::Exchange* lds) {
    float x[8];
    mx::decode8(c, mx::own_scales<false>(s), x);
    if constexpr (!BF16) mx::exchange<true>(*lds, x);
    mx::store_values<BF16, !BF16, WHOLE>(out, at, n, x);
}

template <bool BF16>
__global__ __launch_bounds__(kMxLanes) void mx4_dequantize_kernel(Mx4Args) {
    constexpr int U = kMx4Spans;
    mx::Exchange* const lds = mx::exchange_area<!BF16>();
    const KMx4 a = (KMx4)(__builtin_amdgcn_kernarg_segment_ptr());
    char* const out = a->values[blockIdx.y];
    const char* const codes = a->codes[blockIdx.y];
    const char* const scales = a->scales[blockIdx.y];
    const int64_t n = a->n;
    const uint32_t tiles = a->tiles;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t at = mx::wave_start<U>(tile);
        uint32_t c[U], s[U];
        if (at + U * mx::kMxSpan <= n) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                c[u] = mx::load_codes<true>(codes, at + u * mx::kMxSpan, n);
                s[u] = mx::load_scale<true>(scales, at + u * mx::kMxSpan, n);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) dequantize_span<BF16, true>(c[u], s[u], out, at + u * mx::kMxSpan, n, lds);
        } else {
            for (int64_t i = at; i < n; i += mx::kMxSpan)
                dequantize_span<BF16, false>(mx::load_codes<false>(codes, i, n),
                                             mx::load_scale<false>(scales, i, n), out, i, n, lds);
        }
    }
}

int launch(const void* fn, const Mx4Launch& l, int spans, unsigned lds, const char* what, const char** msg) {
    Mx4Args a{};
    for (int r = 0; r < l.P; ++r) {
        a.values[r] = static_cast<char*>(const_cast<void*>(l.values[r]));
        a.left[r] = static_cast<char*>(l.left[r]);
        a.codes[r] = static_cast<char*>(l.codes[r]);
        a.scales[r] = static_cast<char*>(l.scales[r]);
    }
    a.n = l.n;
    a.tiles = static_cast<uint32_t>(mx_tiles(l.n, spans));
    const unsigned grid = std::min(a.tiles, kMaxMxGrid / static_cast<unsigned>(l.P));
    void* args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3(grid, static_cast<unsigned>(l.P)), dim3(kMxLanes), args, lds,
                                         static_cast<hipStream_t>(l.stream));
    if (e == hipSuccess) return 0;
    *msg = what;
    return static_cast<int>(e);
}

}  // namespace

int launch_mx4_quantize(const Mx4Launch& l, const char** msg) {
#define DDP_KERNELS(BF16, U)                                            \
    {reinterpret_cast<const void*>(&mx4_quantize_kernel<BF16, 0, U>),   \
     reinterpret_cast<const void*>(&mx4_quantize_kernel<BF16, 1, U>),   \
     reinterpret_cast<const void*>(&mx4_quantize_kernel<BF16, 2, U>)}
    const void* const fns[2][2][3] = {{DDP_KERNELS(false, kMx4Spans), DDP_KERNELS(true, kMx4Spans)},
                                      {DDP_KERNELS(false, 1), DDP_KERNELS(true, 1)}};
#undef DDP_KERNELS
    const bool few = l.n <= kMxShort / l.P;
    return launch(fns[few][l.bf16][l.left_type], l, few ? 1 : kMx4Spans,
                  lds_reserve(mx4_quantize_wg_per_cu(l.left_type != 0)), "hipLaunchKernel(mx4_quantize)", msg);
}

int launch_mx4_dequantize(const Mx4Launch& l, const char** msg) {
    const void* const fn = l.bf16 ? reinterpret_cast<const void*>(&mx4_dequantize_kernel<true>)
                                  : reinterpret_cast<const void*>(&mx4_dequantize_kernel<false>);
    return launch(fn, l, kMx4Spans, lds_reserve(mx4_dequantize_wg_per_cu(l.bf16), l.bf16 ? 0 : mx::kExchangeBytes),
                  "hipLaunchKernel(mx4_dequantize)", msg);
}

}  // namespace ddp

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
//
// Bound by HBM: 17/32 byte an element and rank in, 4 or 2 (or 17/32) out for
// each copy, against 1.6 instructions an element and rank.  86.6M elements: 8 ranks
// into one float32 copy 111 us, 6.4 TB/s; with the norm 116, its partials' sum
// 4 of them; 16 ranks coded again with a float32 left-over 233 us, 6.3 TB/s.
//
// Layout (mx.h): codes as they lie, 8 elements a lane, so that a wave decodes 512
// elements with one dword and one byte a rank in each lane, all ranks' loads in
// flight at once; float32 results go through LDS to whole lines (without that,
// 16 bytes of every 32 by an instruction, 125 us; loading codes in the order of
// whole float32 lines instead, which halves what a load's lanes share of a line,
// 157).  A wave with little to load takes more than one span; us for 86.6M elements
// coded again by spans 1, 2, 4 --
//     one copy  P = 2  39 31 26   P = 3  48 38 33   P = 4  47 41 39   P = 6  60 56 57
//               P = 8  70 73 75
//     all       P = 2  43 36 31   P = 3  55 50 52   P = 4  67 70 69   P = 6 101 107 106
//     one copy with a bf16 left-over  P = 2  78 80 80   P = 8  123 129 129
// (to bf16, one copy: P = 2 59 50 51, P = 4 69 64).  Short rows take one: 2 ranks of
// 65,536 coded again 2.8 us with one span, 3.5 with four, of 4.2M 4.0 and 4.3, of
// 8.4M 6.1 and 5.2.  Workgroups of 4 waves keep the 128 bytes of scales that 4,096
// elements have in one or two L2s; one-wave workgroups took 146 us for the first
// case.
//
// One copy runs fastest with the CUs full.  Every rank written as values is
// nearly all writes, many streams at once, and wants fewer: us for 86.6M elements by
// workgroups per CU 0 (full), 1, 2, 3, 4, 5, 6 --
//     float32  P = 2    151  230  164  149  131  125  147
//              P = 3    229  278  237  213  201  226
//              P = 4    314  331  273  274  304  306  308
//              P = 6    477  482  448  459  464  468
//              P = 7    560  515  523  537  543  543
//              P = 8    643  537  602  621  624  632  644
//              P = 16  1305 1209 1234 1273
//     bf16     P = 2     74  130   99   81   73   72   74
//              P = 6    250  303  280  232  226  225
//              P = 7    283  351  326  265  261  278
//              P = 8    326  403  328  306  311  331  331
//              P = 12   490  503  501  475  504  489
//              P = 13   536  517  518  530  553  534
//              P = 16   669  629  665  644  679  656
// and with the norm --
//     float32  P = 2    154  285  217  174  155  138  132
//              P = 3    234  294  267  255  227  200
//              P = 4    318  336  357  274  297  310  312
//              P = 6    484  517  541  460  469  470
//              P = 7    561  515  595  544  553  548
//              P = 8    645  557  561  624  633  632
//              P = 10   813  717  706  788  795  799
//              P = 16  1301 1213 1272 1265 1276 1286
//     bf16     P = 2     78  191  117   98   84   78
//              P = 6    251  423  300  241  231  229
//              P = 8    322  458  363  302  303  311
//              P = 12   495  568  533  480  490  509
//              P = 13   541  584  598  521  552  549
//              P = 16   671  673  685  640  672  653
// The rules in launch_mx.h are within 2% of the best of each row.  Coded again,
// every rank is written two streams of 16 and 1 bytes a block; full CUs are within
// 1% of the best up to 4 ranks, and 2 to 5% above it from 7 on --
//              P = 4     65            120   96   80   71
//              P = 7    114  328  211  159  130  114  112
//              P = 8    133  337  217  164  134  128  127
//              P = 12   201  446  262  216  196  195  196
//              P = 16   275  528  303  271  262  265  269
// (floors at 6.7 TB/s 55, 96, 110, 165, 220).
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
};
typedef const __attribute__((address_space(4))) ReduceArgs* KReduce;

constexpr bool has_f32(int out) { return out == kMxF32 || out == kMxCodedLeftF32; }

// s / P, correctly rounded.  For P no power of two from the product with 1 / P
// and one correction by its remainder, which is exact in a fused multiply-add
// (Markstein's division).  For each of these P that gives the nearest float32 for
// all 2^23 mantissas of s, and so wherever the quotient is normal.  Below, its last
// place is 2^-149 and s, a sum of codes, a multiple of 2^-128: the exact quotient
// is then no tie and at least 1 / 2P of a place from one, the error 2^-24 of that.
// 86.6M elements of 3 ranks coded again took 46 us with this in float64, 38 now.
template <int P>
__device__ __forceinline__ float mean_of(float s) {
    if constexpr ((P & (P - 1)) == 0) {
        return s * (1.0f / static_cast<float>(P));
    } else {
        constexpr float p = P, r = 1.0f / P;
        const float q = s * r;
        const float m = __builtin_fmaf(__builtin_fmaf(-p, q, s), r, q);
        // a zero keeps its sign and an infinity is its own quotient, where the
        // remainder would not know
        constexpr int kOrdinary = 0x198;      // normal or subnormal, of either sign
        return __builtin_amdgcn_classf(s, kOrdinary) ? m : s;
    }
}

template <int P, int OUT, bool WHOLE>
__device__ __forceinline__ void reduce_span(KReduce a, const uint32_t (&c)[P], const uint32_t (&s)[P], const mx::Raw& left,
                                            int64_t at, int64_t n, mx::Exchange* lds, double& sq) {
    float g[8];
    mx::decode8(c[0], mx::own_scales<false>(s[0]), g);
#pragma unroll
    for (int r = 1; r < P; ++r) {
        float x[8];
        mx::decode8(c[r], mx::own_scales<false>(s[r]), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] += x[e];
    }
    if (a->mean) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = mean_of<P>(g[e]);
    }
    if constexpr (OUT >= kMxCoded) {
        float old[8];
        if constexpr (OUT != kMxCoded) {
            float (&x)[8] = old;
            mx::values_of<OUT == kMxCodedLeftBf16, has_f32(OUT)>(left, x);
            if constexpr (has_f32(OUT)) mx::exchange<false>(*lds, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] += x[e];
        }
        if constexpr (!WHOLE) {     // behind the row's end the codes are zero
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!mx::in_row<false>(at, n, e)) g[e] = 0.0f;
        }
        const mx::Coded q = mx::quantize8<false>(g);
        float x[8];
        mx::decode8(q.codes, q.scales, x);
        for (int r = 0; r < a->n_out; ++r)
            mx::store_coded<false, WHOLE>(a->out[r], a->out_scales[r], at, n, q.codes, q.scales);
        if constexpr (OUT != kMxCoded) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = g[e] - x[e];
            if constexpr (has_f32(OUT)) {
                // a block without numbers keeps what it had
                if (!q.finite_a) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = old[e];
                }
                mx::exchange<true>(*lds, y);
                mx::store_values<false, true, WHOLE>(a->left, at, n, y);
            } else {
                mx::store_values<true, false, WHOLE>(a->left, at, n, y, q.finite_a);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = x[e];
    } else {
        if constexpr (has_f32(OUT)) mx::exchange<true>(*lds, g);
        for (int r = 0; r < a->n_out; ++r) mx::store_values<OUT == kMxBf16, has_f32(OUT), WHOLE>(a->out[r], at, n, g);
    }
    if (a->partials != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (WHOLE || mx::in_row<OUT == kMxF32>(at, n, e)) sq = rr::square_to(sq, rr::written<OUT == kMxBf16>(g[e]));
    }
}

template <int P, int OUT, int U>
__global__ __launch_bounds__(kMxLanes) void mx4_reduce_kernel(ReduceArgs) {
    mx::Exchange* const lds = mx::exchange_area<has_f32(OUT)>();
    const KReduce a = (KReduce)(__builtin_amdgcn_kernarg_segment_ptr());
    const int64_t n = a->n;
    const uint32_t tiles = a->tiles;
    double sq = 0.0;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t at = mx::wave_start<U>(tile);
        uint32_t c[U][P], s[U][P];
        mx::Raw left[U];
        if (at + U * mx::kMxSpan <= n) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int r = 0; r < P; ++r) {
                    c[u][r] = mx::load_codes<true>(a->codes[r], at + u * mx::kMxSpan, n);
                    s[u][r] = mx::load_scale<true>(a->scales[r], at + u * mx::kMxSpan, n);
                }
                if constexpr (OUT > kMxCoded)
                    left[u] = mx::load_raw<OUT == kMxCodedLeftBf16, has_f32(OUT), true>(a->left, at + u * mx::kMxSpan, n);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) reduce_span<P, OUT, true>(a, c[u], s[u], left[u], at + u * mx::kMxSpan, n, lds, sq);
        } else {
            for (int64_t i = at; i < n; i += mx::kMxSpan) {
#pragma unroll
                for (int r = 0; r < P; ++r) {
                    c[0][r] = mx::load_codes<false>(a->codes[r], i, n);
                    s[0][r] = mx::load_scale<false>(a->scales[r], i, n);
                }
                if constexpr (OUT > kMxCoded) left[0] = mx::load_raw<OUT == kMxCodedLeftBf16, has_f32(OUT), false>(a->left, i, n);
                reduce_span<P, OUT, false>(a, c[0], s[0], left[0], i, n, lds, sq);
            }
        }
    }
    if (a->partials != nullptr) {
        sq = gv::block_sum<kMxLanes>(sq);
        if (threadIdx.x == 0) {
            a->partials[blockIdx.x] = sq;
            if (blockIdx.x == 0 && a->zero != nullptr) *a->zero = 0;
        }
    }
}

template <int P, int OUT, int U>
const void* kernel_of() {
    if constexpr (U == 1 || U == mx4_reduce_spans(P, OUT, true) || U == mx4_reduce_spans(P, OUT, false))
        return reinterpret_cast<const void*>(&mx4_reduce_kernel<P, OUT, U>);
    else
        return nullptr;
}
template <int OUT>
const void* kernel_for(int P, int spans) {
    switch (P) {
#define DDP_CASE(p) \
    case p:         \
        return spans == 1 ? kernel_of<p, OUT, 1>() : spans == 2 ? kernel_of<p, OUT, 2>() : kernel_of<p, OUT, 4>();
        DDP_CASE(1) DDP_CASE(2) DDP_CASE(3) DDP_CASE(4)
        DDP_CASE(5) DDP_CASE(6) DDP_CASE(7) DDP_CASE(8)
        DDP_CASE(9) DDP_CASE(10) DDP_CASE(11) DDP_CASE(12)
        DDP_CASE(13) DDP_CASE(14) DDP_CASE(15) DDP_CASE(16)
#undef DDP_CASE
        default:
            return nullptr;
    }
}

// LDS that lets so many workgroups share a CU, beside what the kernel has of its
// own (the exchange, and the norm's four sums).
unsigned lds_for(int wg_per_cu, bool f32) {
    const unsigned own = (f32 ? mx::kExchangeBytes : 0) + (kMxLanes / 64) * sizeof(double);
    if (wg_per_cu == 1) return kLdsBytesPerCu / 2;      // with its own, more than half
    return lds_reserve(wg_per_cu, own);
}

}  // namespace

int launch_mx4_reduce(const Mx4Reduce& l, int64_t* workgroups, const char** msg) {
    ReduceArgs a{};
    for (int r = 0; r < l.P; ++r) {
        a.codes[r] = static_cast<const char*>(l.codes[r]);
        a.scales[r] = static_cast<const char*>(l.scales[r]);
    }
    for (int r = 0; r < l.n_out; ++r) {
        a.out[r] = static_cast<char*>(l.out[r]);
        a.out_scales[r] = static_cast<char*>(l.out_scales[r]);
    }
    const bool coded = l.out_type == kMxCoded;
    const int out = l.out_type + (coded ? l.left_type : 0);
    const bool f32 = has_f32(out);
    const int spans = l.n <= kMxOneSpan ? 1 : mx4_reduce_spans(l.P, out, l.n_out == 1);
    a.left = static_cast<char*>(l.left);
    a.partials = l.partials;
    a.zero = l.zero;
    a.n = l.n;
    a.tiles = static_cast<uint32_t>(mx_tiles(l.n, spans));
    a.n_out = l.n_out;
    a.mean = l.mean;
    const void* fn = out == kMxF32 ? kernel_for<kMxF32>(l.P, spans) : out == kMxBf16 ? kernel_for<kMxBf16>(l.P, spans)
                     : out == kMxCoded ? kernel_for<kMxCoded>(l.P, spans)
                     : out == kMxCodedLeftF32 ? kernel_for<kMxCodedLeftF32>(l.P, spans)
                                              : kernel_for<kMxCodedLeftBf16>(l.P, spans);
    const unsigned grid = std::min(a.tiles, kMaxMxGrid);
    *workgroups = grid;
    void* args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3(grid), dim3(kMxLanes), args,
                                         lds_for(mx4_reduce_wg_per_cu(l.P, f32, l.n_out > 1 && !coded, l.partials != nullptr), f32),
                                         static_cast<hipStream_t>(l.stream));
    if (e == hipSuccess) return 0;
    *msg = "hipLaunchKernel(mx4_reduce)";
    return static_cast<int>(e);
}

}  // namespace ddp

// Launch interface of the 4-bit gradient and 8-bit moment kernels (mx4.hip,
// mx4_reduce.hip, adamw8.hip) between api.cpp and the kernels.  Internal, like
// launch.h.
#pragma once

#include "launch_grads.h"

namespace ddp {

constexpr int64_t mx_blocks(int64_t n) { return n / DDP_MX_BLOCK + (n % DDP_MX_BLOCK != 0); }

// The 4-bit kernels' workgroups: 4 waves, each taking so many spans of 512
// elements.
constexpr unsigned kMxLanes = 256;
constexpr int64_t mx_tiles(int64_t n, int spans) { return (n + 2048 * spans - 1) / (2048 * spans); }
// A grid holds fewer than 2^32 lanes; each workgroup walks on by its size.
constexpr uint32_t kMaxMxGrid = 1u << 23;

// Elements up to which a launch's waves take one span each, not two: a short one
// ends no sooner than its longest wave (figures in mx4.hip and adamw8.hip).
constexpr int64_t kMxShort = 1 << 20;

// Quantisation and reading back: spans per wave, and workgroups per CU (figures
// in mx4.hip).
constexpr int kMx4Spans = 2;
constexpr int mx4_quantize_wg_per_cu(bool left) { return left ? 4 : 6; }
constexpr int mx4_dequantize_wg_per_cu(bool bf16) { return bf16 ? 5 : 4; }

// What the all-reduce writes: values, or codes with the left-over as the last
// word has it.
enum Mx4Out { kMxF32 = 0, kMxBf16 = 1, kMxCoded = 2, kMxCodedLeftF32 = 3, kMxCodedLeftBf16 = 4 };
// The all-reduce (figures in mx4_reduce.hip).  Spans per wave on long rows: more
// than one where a span moves little, few ranks and neither float32 nor a
// left-over; `one`: into one copy.
constexpr int mx4_reduce_spans(int P, int out, bool one) {
    if (out == kMxBf16) return P <= 4 ? 2 : 1;
    if (out != kMxCoded) return 1;
    if (one) return P <= 4 ? 4 : P <= 7 ? 2 : 1;
    return P <= 2 ? 4 : P <= 3 ? 2 : 1;
}
// One while the waves of all spans fit the GPU at once.
constexpr int64_t kMxOneSpan = 1 << 22;
// Workgroups per CU, 0 for no limit: fewer the more every rank receives as
// values, but not where the waves wait for the norm's sums: up to 6 ranks one more
// for float32 (from 7 on one is best with the norm too), for bf16 no fewer than 3.
constexpr int mx4_reduce_wg_per_cu(int P, bool f32, bool all_ranks_values, bool norm) {
    if (!all_ranks_values) return 0;
    if (!f32) return P <= 6 ? 5 : P <= 12 || norm ? 3 : 1;
    if (P > 6) return 1;
    return (P <= 2 ? 5 : P <= 3 ? 4 : 2) + (norm ? 1 : 0);
}

// The AdamW step with 8-bit moments and their reading back (adamw8.hip).
constexpr int kAdamW8WgPerCu = 4;
constexpr int kMoments8WgPerCu = 3;

// P rows between values and codes.
struct Mx4Launch {
    int P;
    int64_t n;
    const void* values[kMaxRanks];   // quantise: the input; dequantise: the output
    int bf16;
    void* left[kMaxRanks];           // quantise: the left-over, read and written
    int left_type;                   // 0 none, 1 float32, 2 bf16
    void* codes[kMaxRanks];
    void* scales[kMaxRanks];
    void* stream;
};
int launch_mx4_quantize(const Mx4Launch& l, const char** msg);
int launch_mx4_dequantize(const Mx4Launch& l, const char** msg);

// The all-reduce of P coded rows.
struct Mx4Reduce {
    int P;
    int mean;
    int64_t n;
    const void* codes[kMaxRanks];
    const void* scales[kMaxRanks];
    int n_out;
    int out_type;                    // Mx4Out without a left-over
    void* out[kMaxRanks];            // coded: the codes
    void* out_scales[kMaxRanks];
    void* left;
    int left_type;
    double* partials;                // one per workgroup, or null: no norm
    uint64_t* zero;                  // cleared by the first workgroup, or null
    void* stream;
};
// Also tells how many workgroups it started, and so partials it leaves.
int launch_mx4_reduce(const Mx4Reduce& l, int64_t* workgroups, const char** msg);
// Workgroups, and so partials, of such a launch at most.
constexpr int64_t mx4_reduce_partials(int64_t n) {
    return mx_tiles(n, 1) < kMaxMxGrid ? mx_tiles(n, 1) : static_cast<int64_t>(kMaxMxGrid);
}

// One AdamW step with 8-bit moments on n_tensors tensors.
struct AdamW8Launch {
    AdamWLaunch step;                // m and v unused
    uint8_t* const* m;
    uint8_t* const* v;
    uint8_t* const* scales;
    int64_t seed;
};
int launch_adamw8(const AdamW8Launch& l, const char** msg);

// 8-bit moments as values.
struct Moments8Read {
    int32_t n_tensors;
    const int64_t* numels;
    const uint8_t* const* m;
    const uint8_t* const* v;
    const uint8_t* const* scales;
    void* const* m_out;
    void* const* v_out;
    int out_bf16;
    void* stream;
};
int launch_adamw8_read(const Moments8Read& l, const char** msg);

}  // namespace ddp

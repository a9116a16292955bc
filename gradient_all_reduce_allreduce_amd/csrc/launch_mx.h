// Launch interface of the 4-bit gradient and 8-bit moment kernels (mx4.hip,
// mx4_reduce.hip, adamw8.hip) between api.cpp and the kernels.  Internal, like
// launch.h.
#pragma once

#include "launch_grads.h"

namespace ddp {

constexpr int64_t mx_blocks(int64_t n) { return n / DDP_MX_BLOCK + (n % DDP_MX_BLOCK != 0); }

// Elements per one-wave workgroup of the 4-bit kernels: 8 per lane.
constexpr int64_t kMxTileElems = 512;
constexpr int64_t mx_tiles(int64_t n) { return n / kMxTileElems + (n % kMxTileElems != 0); }

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
    int out_type;                    // 0 float32, 1 bf16, 2 coded
    void* out[kMaxRanks];            // coded: the codes
    void* out_scales[kMaxRanks];
    void* left;
    int left_type;
    double* partials;                // one per workgroup, or null: no norm
    uint64_t* zero;                  // cleared by the first workgroup, or null
    void* stream;
};
int launch_mx4_reduce(const Mx4Reduce& l, const char** msg);
// Workgroups of that launch, and so its partials.
int64_t mx4_reduce_workgroups(int64_t n);

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

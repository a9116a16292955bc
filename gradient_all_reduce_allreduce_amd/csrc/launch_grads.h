// Launch interface of the gradient norm, clipping and AdamW kernels
// (grad_norm.hip, adamw.hip) between api.cpp and the kernels.  Internal,
// like launch.h.
#pragma once

#include <stddef.h>

#include "launch.h"

namespace ddp {

// Kernel arguments that carry the tensors' addresses stay under the 8,000
// bytes measured to pass.
constexpr size_t kArgBytes = 7936;
// A longer tensor goes as several pieces of so many elements (a multiple of
// a line for every type), so that a kernel counts elements in 32 bits.
constexpr int64_t kMaxPiece = int64_t(1) << 30;
// One-wave workgroups of a launch at most (a grid holds fewer than 2^32
// lanes); each walks on by the grid's size.
constexpr uint32_t kMaxWaveGrid = 1u << 25;

// Partial sums a norm leaves in its workspace at most, one per workgroup:
// 4 workgroups of 256 lanes per CU.
constexpr int kNormPartials = DDP_NORM_WORKSPACE_BYTES / static_cast<int>(sizeof(double));
// Up to so many 4 KiB tiles, a tensor's first and last counting as one each:
// one workgroup takes the norm, and scales, in one launch.
constexpr int kSmallTiles = 64;
// One-wave workgroups of the scaling per CU, the fastest of 12, 14, 16, 20, 24
// and no cap by up to 4%.
constexpr int kClipWgPerCu = 12;

// The global norm of n_tensors gradient tensors, and their scaling.
struct NormLaunch {
    int32_t n_tensors;
    const int64_t* numels;
    const void* const* in;
    const int32_t* dtypes;    // ddp_dtype of each tensor
    void* const* out;         // clip: where the scaled tensors go; else null
    bool norm_given;
    double* partials;         // [kNormPartials], device; null: small, or the norm is given
    float* norm;              // device: the norm, written or (given) read
    float max_norm;
    void* stream;
};
// Whether these take the one-workgroup path, which needs no partials.
bool norm_is_small(int32_t n_tensors, const int64_t* numels, const void* const* in, const int32_t* dtypes);
int launch_norm(const NormLaunch& l, const char** msg);
// out = in * min(1, max_norm / (norm + 1e-6)), the norm taken first unless
// it is given.
int launch_clip(const NormLaunch& l, const char** msg);

// norm = sqrt(sum of count partials).  More than kNormFoldOver of them are
// summed by kNormFold workgroups through `fold` (not touched otherwise):
// kNormFold sums and a count that is zero when this launch starts.  On
// 99,832 partials (P = 8, 25.6M elements) 64 workgroups of 1,024 lanes add 3.7
// us to the all-reduce, 256 of 256 lanes 7.7 us (each of them takes a turn
// at the count) and one of 1,024 lanes 26 us; an empty launch adds 1.6 us.
// On 4,000 partials one workgroup and 64 take the same.
constexpr int64_t kNormFoldOver = 4096;
constexpr int kNormFold = 64;
int launch_norm_of(const double* partials, int64_t count, double* fold, float* norm, void* stream, const char** msg);

// One-wave workgroups of the AdamW step per CU (figures in adamw.hip): the best
// or within 2% of it for every pair of types.
constexpr int kAdamWWgPerCu = 12;

// One AdamW step on n_tensors tensors.
struct AdamWLaunch {
    int32_t n_tensors;
    const int64_t* numels;
    const void* const* grads;
    float* const* w;
    float* const* m;
    float* const* v;
    void* const* params;      // may be null
    int grad_bf16;
    int param_bf16;
    double lr;
    double beta1;
    double beta2;
    double eps;
    double weight_decay;
    int64_t step;
    const int64_t* step_dev;  // null: `step`
    const float* norm;        // null: no clipping
    float max_norm;
    void* stream;
};
int launch_adamw(const AdamWLaunch& l, const char** msg);

}  // namespace ddp

// Launch interface of the gradient norm, clipping and AdamW kernels
// (grad_norm.hip, adamw.hip) between api.cpp and the kernels.  Internal,
// like launch.h.
#pragma once

#include "launch.h"

namespace ddp {

// Partial sums a norm leaves in its workspace at most, one per workgroup.
constexpr int kNormPartials = DDP_NORM_WORKSPACE_BYTES / static_cast<int>(sizeof(double));

// The global norm of n_tensors gradient tensors, and their scaling.
struct NormLaunch {
    int32_t n_tensors;
    const int64_t* numels;
    const void* const* in;
    const int32_t* dtypes;    // ddp_dtype of each tensor
    void* const* out;         // clip: where the scaled tensors go
    double* partials;         // [kNormPartials], device; null when the norm is given
    float* norm;              // device: the norm, written (partials) or read
    float max_norm;
    void* stream;
};

// The squares' sums of every tensor into l.partials; *n_partials of them.
int launch_square_sums(const NormLaunch& l, int* n_partials, const char** msg);
// norm = sqrt(sum of count partials); more than kNormFoldOver of them are
// first folded to kNormFold in `fold` (not read otherwise).
constexpr int64_t kNormFoldOver = 16384;
constexpr int kNormFold = 512;
int launch_norm_of(const double* partials, int64_t count, double* fold, float* norm, void* stream, const char** msg);
// out = in * min(1, max_norm / (norm + 1e-6)); with partials (n_partials of
// them) the norm is their root and is written to l.norm too.
int launch_clip(const NormLaunch& l, int n_partials, const char** msg);

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

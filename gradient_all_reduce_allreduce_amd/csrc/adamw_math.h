// adamw_math.h -- the AdamW step on one element and the factors that are the
// same for all of them, shared by the steps with 32-bit and with 8-bit moments
// (adamw.hip, adamw8.hip).
//
// With c = min(1, max_norm / (norm + 1e-6)) (1 without a norm), t the step's
// number from 1, and per element, float32 with one rounding per operation:
//     g = c * g
//     m = b1 * m + (1 - b1) * g
//     v = b2 * v + (1 - b2) * (g * g)
//     w = w * (1 - lr * wd) - lr / (1 - b1^t) * (m / (sqrt(v) / sqrt(1 - b2^t) + eps))
// The factors that are the same for every element (1 - b1, 1 - lr * wd,
// lr / (1 - b1^t), 1 / sqrt(1 - b2^t)) are computed in float64 and rounded to
// float32 once: 1 - b2 taken in float32 would be off by 5e-5 for b2 = 0.999.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grad_vec.h"
#include "launch_grads.h"

namespace ddp {
namespace adamw {

// The step's scalars as kernel arguments.
struct Scalars {
    const float* norm;
    const int64_t* step;     // device; null: host_step, and step_size and root2 hold its factors
    int64_t host_step;
    double b1, b2, lr;       // with `step`
    float max_norm;
    float beta1, beta2;
    float one_beta1, one_beta2;
    float decay;
    float eps;
    float step_size;
    float root2;
};
typedef const __attribute__((address_space(4))) Scalars* KScalars;

// What depends on the step's number: lr / (1 - b1^t) and 1 / sqrt(1 - b2^t),
// the powers by squaring, all float64, rounded to float32 once.
struct StepFactors {
    float size, root2;
};
inline StepFactors step_factors(double lr, double b1, double b2, int64_t t) {
    double p1 = 1.0, p2 = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) {
            p1 *= b1;
            p2 *= b2;
        }
        b1 *= b1;
        b2 *= b2;
    }
    return {static_cast<float>(lr / (1.0 - p1)), static_cast<float>(1.0 / __builtin_sqrt(1.0 - p2))};
}

// The same on the GPU, the same for the whole wave: even lanes work out the
// first of the two, odd lanes the second, with the same operations on each.
__device__ __forceinline__ StepFactors wave_step_factors(double lr, double b1, double b2, int64_t t) {
    const bool odd = threadIdx.x & 1;
    double b = odd ? b2 : b1, p = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) p *= b;
        b *= b;
    }
    const double rest = 1.0 - p;
    const float x = static_cast<float>((odd ? 1.0 : lr) / (odd ? __builtin_sqrt(rest) : rest));
    const int f = static_cast<int>(__float_as_uint(x));
    return {__uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(f, 0))),
            __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(f, 1)))};
}

inline Scalars scalars_of(const AdamWLaunch& l) {
    Scalars a;
    a.norm = l.norm;
    a.max_norm = l.max_norm;
    a.step = l.step_dev;
    a.host_step = l.step;
    a.b1 = l.beta1;
    a.b2 = l.beta2;
    a.lr = l.lr;
    a.beta1 = static_cast<float>(l.beta1);
    a.beta2 = static_cast<float>(l.beta2);
    a.one_beta1 = static_cast<float>(1.0 - l.beta1);
    a.one_beta2 = static_cast<float>(1.0 - l.beta2);
    a.decay = static_cast<float>(1.0 - l.lr * l.weight_decay);
    a.eps = static_cast<float>(l.eps);
    a.step_size = 0.0f;
    a.root2 = 0.0f;
    if (l.step_dev == nullptr) {
        const StepFactors s = step_factors(l.lr, l.beta1, l.beta2, l.step);
        a.step_size = s.size;
        a.root2 = s.root2;
    }
    return a;
}

struct Factors {
    float c, beta1, beta2, one_beta1, one_beta2, decay, eps, step_size, root2;
};

__device__ __forceinline__ void adamw_moments(float g, float& m, float& v, const Factors& f) {
#pragma clang fp contract(off)
    g = g * f.c;
    const float m0 = f.beta1 * m;
    const float m1 = f.one_beta1 * g;
    m = m0 + m1;
    const float v0 = f.beta2 * v;
    const float gg = g * g;
    const float v1 = f.one_beta2 * gg;
    v = v0 + v1;
}

__device__ __forceinline__ void adamw_element(float g, float& w, float& m, float& v, const Factors& f) {
#pragma clang fp contract(off)
    adamw_moments(g, m, v, f);
    const float r = __builtin_sqrtf(v) * f.root2;
    const float d = r + f.eps;
    const float q = m / d;
    const float w0 = w * f.decay;
    const float s = f.step_size * q;
    w = w0 - s;
}

// The factors from the arguments and the norm and step count they point to.
// False: the step is left out.
__device__ __forceinline__ bool factors(KScalars a, float norm, int64_t t, Factors& f) {
    f.c = 1.0f;
    if (a->norm != nullptr) {
        if (!(__builtin_fabsf(norm) < __builtin_inff())) return false;
        f.c = gv::clip_factor(norm, a->max_norm);
    }
    f.step_size = a->step_size;
    f.root2 = a->root2;
    if (a->step != nullptr) {
        if (t < 1) return false;
        const StepFactors s = wave_step_factors(a->lr, a->b1, a->b2, t);
        f.step_size = s.size;
        f.root2 = s.root2;
    }
    f.beta1 = a->beta1;
    f.beta2 = a->beta2;
    f.one_beta1 = a->one_beta1;
    f.one_beta2 = a->one_beta2;
    f.decay = a->decay;
    f.eps = a->eps;
    return true;
}

}  // namespace adamw
}  // namespace ddp

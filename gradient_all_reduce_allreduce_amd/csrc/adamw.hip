// adamw.hip -- one AdamW step on many tensors, the gradient clipped on the
// way, for gfx950.
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
// w, m and v are float32 and updated in place; a copy of the new weights
// goes out as float32 or bf16 (nearest even).  A norm that is not finite
// leaves everything as it was.
//
// Bound by HBM: gradient, w, m and v are read once and w, m, v and the copy
// written once (28 bytes an element with bf16 gradient and copy), against some
// forty instructions, a correctly rounded division and square root among them.
// 86.6M elements, bf16 gradient and copy: 370 us, 6.5 TB/s; 658M: 2.79 ms, 6.6.
//
// Layout: one one-wave workgroup per tile of 256 elements, a tile starting on
// a line of w (a tensor's first one is short when its w starts inside a line),
// every lane 4 consecutive elements of each stream; the other streams usually
// lie the same way and are read as they lie if not.  With as many workgroups as
// tiles and few of them on a CU the mix of four streams in and four out moves
// as the all-reduce's does (launch.h): workgroups of 256 that walk over many
// tiles took 492 us instead of 370, and by the cap on one-wave workgroups per CU
// 8: 421, 10: 381, 12: 373, 14: 382, 16: 381, 20: 400, none: 394 us.
// A new workgroup's way to its first load is the search for its tensor and one
// batch of scalar loads; what the step needs besides (the norm, the step's
// number, divisions, two powers) is worked out while the data is in flight.
// (The norm and the count read as vector loads waited for the tile's data first:
// 463 us with the count on the GPU, 372 now.)  Addresses and sizes travel in
// the kernel arguments, several launches for more tensors than fit.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "grad_vec.h"
#include "launch_grads.h"

namespace ddp {
namespace {

using rr::u32x2;
using rr::u32x4;

constexpr int kBlock = 64;                             // one wave
constexpr uint32_t kTileElems = kBlock * 4;
constexpr uint32_t kLineElems = 32;                    // float32 per 128-byte line
// Tensors (or pieces of them) per launch: as many as the arguments hold.
// (Arguments for 16 only, for calls with so few, made no difference.)
constexpr int kCap = 162;

struct AdamWArgs {
    const char* g[kCap];
    char* w[kCap];
    char* m[kCap];
    char* v[kCap];
    char* p[kCap];
    uint32_t count[kCap];     // elements, up to kMaxPiece
    uint32_t first_tile[kCap];
    int32_t n;
    uint32_t tiles;          // of all pieces
    const float* norm;
    const int64_t* step;     // device; null: step_size and root2 hold the step's
    double b1, b2, lr;       // with `step`
    float max_norm;
    float beta1, beta2;
    float one_beta1, one_beta2;
    float decay;
    float eps;
    float step_size;
    float root2;
};
static_assert(sizeof(AdamWArgs) <= kArgBytes, "kernel arguments");
typedef const __attribute__((address_space(4))) AdamWArgs* KAdamW;

// What depends on the step's number: lr / (1 - b1^t) and 1 / sqrt(1 - b2^t),
// the powers by squaring, all float64, rounded to float32 once.
struct StepFactors {
    float size, root2;
};
__host__ __device__ __forceinline__ StepFactors step_factors(double lr, double b1, double b2, int64_t t) {
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

struct Factors {
    float c, beta1, beta2, one_beta1, one_beta2, decay, eps, step_size, root2;
};

__device__ __forceinline__ void adamw_element(float g, float& w, float& m, float& v, const Factors& f) {
#pragma clang fp contract(off)
    g = g * f.c;
    const float m0 = f.beta1 * m;
    const float m1 = f.one_beta1 * g;
    m = m0 + m1;
    const float v0 = f.beta2 * v;
    const float gg = g * g;
    const float v1 = f.one_beta2 * gg;
    v = v0 + v1;
    const float r = __builtin_sqrtf(v) * f.root2;
    const float d = r + f.eps;
    const float q = m / d;
    const float w0 = w * f.decay;
    const float s = f.step_size * q;
    w = w0 - s;
}

// The factors from the arguments and the norm and step count they point to.
// False: the step is left out.
__device__ __forceinline__ bool factors(KAdamW a, float norm, int64_t t, Factors& f) {
    f.c = 1.0f;
    if (a->norm != nullptr) {
        if (!(__builtin_fabsf(norm) < __builtin_inff())) return false;
        f.c = gv::clip_factor(norm, a->max_norm);
    }
    f.step_size = a->step_size;
    f.root2 = a->root2;
    if (a->step != nullptr) {
        if (t < 1) return false;
        const StepFactors s = step_factors(a->lr, a->b1, a->b2, t);
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

// GB: bf16 gradients.  PM: the copy, 0 none, 1 float32, 2 bf16.
template <bool GB, int PM>
__global__ __launch_bounds__(kBlock) void adamw_kernel(AdamWArgs) {
    const KAdamW a = (KAdamW)(__builtin_amdgcn_kernarg_segment_ptr());
    const uint32_t tiles = a->tiles;
    const float norm = a->norm != nullptr ? gv::load_uniform(a->norm) : 0.0f;
    const int64_t step = a->step != nullptr ? gv::load_uniform(a->step) : 1;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        int t = 0;
        for (int h = a->n - 1; t < h;) {
            const int mid = (t + h + 1) >> 1;
            if (a->first_tile[mid] <= tile) t = mid; else h = mid - 1;
        }
        const char* const g = a->g[t];
        char* const w = a->w[t];
        char* const m = a->m[t];
        char* const v = a->v[t];
        char* const p = a->p[t];
        const int32_t n = static_cast<int32_t>(a->count[t]);
        const int32_t lead = static_cast<int32_t>((reinterpret_cast<uint64_t>(w) >> 2) % kLineElems);
        const int32_t at = static_cast<int32_t>((tile - a->first_tile[t]) * kTileElems) - lead;
        const int64_t i = at + static_cast<int32_t>(threadIdx.x * 4);
        const bool whole = (at >= 0 && at + static_cast<int32_t>(kTileElems) <= n) || (i >= 0 && i + 4 <= n);
        u32x4 gq, wq, mq, vq;
        if (whole) {
            if constexpr (GB) {
                const u32x2 h = gv::load2_nt(g + i * 2);
                gq = u32x4{h[0], h[1], 0u, 0u};
            } else {
                gq = gv::load4_nt(g + i * 4);
            }
            wq = gv::load4_nt(w + i * 4);
            mq = gv::load4_nt(m + i * 4);
            vq = gv::load4_nt(v + i * 4);
        } else {   // over a tensor's ends
            gq = gv::load_some<GB, 4>(g, i, n);
            wq = gv::load_some<false, 4>(w, i, n);
            mq = gv::load_some<false, 4>(m, i, n);
            vq = gv::load_some<false, 4>(v, i, n);
        }
        // The factors (divisions, two powers) while the tile's data is in
        // flight.
        Factors f;
        if (!factors(a, norm, step, f)) return;
        float wn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float me = __uint_as_float(mq[e]);
            float ve = __uint_as_float(vq[e]);
            wn[e] = __uint_as_float(wq[e]);
            adamw_element(rr::elem<GB>(gq, e), wn[e], me, ve, f);
            wq[e] = __float_as_uint(wn[e]);
            mq[e] = __float_as_uint(me);
            vq[e] = __float_as_uint(ve);
        }
        const u32x2 h = {rr::bf16_bits(wn[0]) | (rr::bf16_bits(wn[1]) << 16),
                         rr::bf16_bits(wn[2]) | (rr::bf16_bits(wn[3]) << 16)};
        if (whole) {
            gv::store4_nt(w + i * 4, wq);
            gv::store4_nt(m + i * 4, mq);
            gv::store4_nt(v + i * 4, vq);
            if constexpr (PM == 1) gv::store4_nt(p + i * 4, wq);
            if constexpr (PM == 2) gv::store2_nt(p + i * 2, h);
        } else {
            gv::store_some<false, 4>(w, i, n, wq);
            gv::store_some<false, 4>(m, i, n, mq);
            gv::store_some<false, 4>(v, i, n, vq);
            if constexpr (PM == 1) gv::store_some<false, 4>(p, i, n, wq);
            if constexpr (PM == 2) gv::store_some<true, 4>(p, i, n, u32x4{h[0], h[1], 0u, 0u});
        }
    }
}

const void* kernel_for(const AdamWLaunch& l) {
    const int pm = l.params == nullptr ? 0 : (l.param_bf16 ? 2 : 1);
    if (l.grad_bf16) {
        return pm == 0 ? reinterpret_cast<const void*>(&adamw_kernel<true, 0>)
               : pm == 1 ? reinterpret_cast<const void*>(&adamw_kernel<true, 1>)
                         : reinterpret_cast<const void*>(&adamw_kernel<true, 2>);
    }
    return pm == 0 ? reinterpret_cast<const void*>(&adamw_kernel<false, 0>)
           : pm == 1 ? reinterpret_cast<const void*>(&adamw_kernel<false, 1>)
                     : reinterpret_cast<const void*>(&adamw_kernel<false, 2>);
}

}  // namespace

int launch_adamw(const AdamWLaunch& l, const char** msg) {
    AdamWArgs a;
    a.norm = l.norm;
    a.max_norm = l.max_norm;
    a.step = l.step_dev;
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
    const void* fn = kernel_for(l);
    int64_t at = 0;   // element of tensor t that the next piece starts at
    for (int32_t t = 0; t < l.n_tensors;) {
        int64_t tiles = 0;
        for (a.n = 0; t < l.n_tensors && a.n < kCap;) {
            const int64_t count = std::min(l.numels[t] - at, kMaxPiece);
            if (count > 0) {
                const int64_t ges = l.grad_bf16 ? 2 : 4;
                const int64_t pes = l.param_bf16 ? 2 : 4;
                a.g[a.n] = static_cast<const char*>(l.grads[t]) + at * ges;
                a.w[a.n] = reinterpret_cast<char*>(l.w[t] + at);
                a.m[a.n] = reinterpret_cast<char*>(l.m[t] + at);
                a.v[a.n] = reinterpret_cast<char*>(l.v[t] + at);
                a.p[a.n] = l.params != nullptr ? static_cast<char*>(l.params[t]) + at * pes : nullptr;
                a.count[a.n] = static_cast<uint32_t>(count);
                a.first_tile[a.n] = static_cast<uint32_t>(tiles);
                const int64_t lead = static_cast<int64_t>((reinterpret_cast<uintptr_t>(a.w[a.n]) >> 2) % kLineElems);
                tiles += (lead + count + kTileElems - 1) / kTileElems;
                at += count;
                ++a.n;
            }
            if (at >= l.numels[t]) {
                ++t;
                at = 0;
            }
        }
        if (a.n == 0) continue;
        a.tiles = static_cast<uint32_t>(tiles);
        const unsigned grid = std::min(a.tiles, kMaxWaveGrid);
        void* args[] = {&a};
        const hipError_t e = hipLaunchKernel(fn, dim3(grid), dim3(kBlock), args, lds_reserve(kAdamWWgPerCu),
                                             static_cast<hipStream_t>(l.stream));
        if (e != hipSuccess) {
            *msg = "hipLaunchKernel(adamw)";
            return static_cast<int>(e);
        }
    }
    return 0;
}

}  // namespace ddp

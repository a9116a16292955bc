// adamw.hip -- one AdamW step on many tensors, the gradient clipped on the
// way, for gfx950.
//
// The mathematics of an element stand in adamw_math.h.
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

#include "adamw_math.h"

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
    adamw::Scalars scalars;
};
static_assert(sizeof(AdamWArgs) <= kArgBytes, "kernel arguments");
typedef const __attribute__((address_space(4))) AdamWArgs* KAdamW;

// GB: bf16 gradients.  PM: the copy, 0 none, 1 float32, 2 bf16.
template <bool GB, int PM>
__global__ __launch_bounds__(kBlock) void adamw_kernel(AdamWArgs) {
    const KAdamW a = (KAdamW)(__builtin_amdgcn_kernarg_segment_ptr());
    const uint32_t tiles = a->tiles;
    const adamw::KScalars k = (adamw::KScalars)(&a->scalars);
    const float norm = k->norm != nullptr ? gv::load_uniform(k->norm) : 0.0f;
    const int64_t step = k->step != nullptr ? gv::load_uniform(k->step) : 1;
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
        adamw::Factors f;
        if (!adamw::factors(k, norm, step, f)) return;
        float wn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float me = __uint_as_float(mq[e]);
            float ve = __uint_as_float(vq[e]);
            wn[e] = __uint_as_float(wq[e]);
            adamw::adamw_element(rr::elem<GB>(gq, e), wn[e], me, ve, f);
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
    a.scalars = adamw::scalars_of(l);
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

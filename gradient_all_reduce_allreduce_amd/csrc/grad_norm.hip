// grad_norm.hip -- the global 2-norm of many gradient tensors and their
// clipping, for gfx950.
//
//     N = sqrt(sum over tensors and elements of g^2)
//     g <- g * min(1, max_norm / (N + 1e-6))
//
// Numbers.  The square of a float32 (or bf16) value is exact in float64 (24
// + 24 bits of 53) and neither overflows nor underflows there, so squares
// and sums are float64 throughout and the norm is rounded to float32 once.
// The sums' order is fixed by the tensors' sizes: workgroup b sums its own
// run of tiles and leaves one partial, and the partials are added in order.
// No atomics: the same tensors give the same bits every time.
//
// Layout.  A tile is 16 KiB of one tensor, its start on a 128-byte line: the
// first tile of a tensor that starts inside a line is short by that much, so
// that a wave's accesses cover whole lines for any start.  Every workgroup
// takes one contiguous run of tiles, finds its tensor once and walks on.
// The tensors' addresses and sizes travel in the kernel arguments (checked on
// the host, nothing on the device that could go stale); more tensors than
// one launch's arguments hold go out as several launches, the later ones
// adding to the partials of the earlier.
//
// Bound by HBM: the norm reads every element once, the scaling reads and
// writes it once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "grad_vec.h"
#include "launch_grads.h"

namespace ddp {
namespace {

using rr::square_to;
using rr::u32x4;

constexpr int kBlock = 256;
constexpr int kVecPerLane = 4;                                       // 16-byte vectors per lane and tile
constexpr uint32_t kTileBytes = kBlock * kVecPerLane * 16;
constexpr uint32_t kLine = 128;
constexpr int64_t kMaxTiles = int64_t(1) << 30;                      // tiles per launch

// The tensors of one launch.  numel's top bit says bf16.
template <int CAP, bool OUT>
struct SetArgs {
    const char* in[CAP];
    char* out[OUT ? CAP : 1];
    uint64_t numel[CAP];
    uint32_t first_tile[CAP + 1];   // first_tile[n] = the number of tiles
    int32_t n;                      // tensors, 1 .. CAP
    int32_t n_partials;             // clip: partials to sum, 0 = the norm is given
    int32_t add;                    // norm: add to the partials already there
    int32_t in_place;               // clip: every output is its input
    double* partials;
    float* norm;
    float max_norm;
    int32_t write_norm;             // clip: this launch writes the norm
};
constexpr uint64_t kBf16Bit = uint64_t(1) << 63;
constexpr int kNormCap = 380;
constexpr int kClipCap = 272;
typedef SetArgs<kNormCap, false> NormArgs;
typedef SetArgs<kClipCap, true> ClipArgs;
static_assert(sizeof(NormArgs) <= 7800 && sizeof(ClipArgs) <= 7800,
              "kernel arguments must stay under the 8,000 bytes measured to pass");

template <class A>
using Konst = const __attribute__((address_space(4))) A*;

// A workgroup's run of tiles and the tensor it is in.  All uniform.
template <class A>
struct Walk {
    Konst<A> a;
    uint32_t tile, last;    // tiles [tile, last)
    int t;
    const char* base;       // the tensor's start, down to a line
    uint64_t lo, hi;        // its bytes [lo, hi) from there
    bool bf16;

    __device__ __forceinline__ explicit Walk(Konst<A> args) : a(args) {
        const uint64_t tiles = a->first_tile[a->n];
        tile = static_cast<uint32_t>(tiles * blockIdx.x / gridDim.x);
        last = static_cast<uint32_t>(tiles * (blockIdx.x + 1) / gridDim.x);
        int l = 0, h = a->n - 1;
        while (l < h) {
            const int mid = (l + h + 1) >> 1;
            if (a->first_tile[mid] <= tile) l = mid; else h = mid - 1;
        }
        t = l;
        enter();
    }
    __device__ __forceinline__ void enter() {
        const uint64_t p = reinterpret_cast<uint64_t>(a->in[t]);
        const uint64_t n = a->numel[t];
        bf16 = (n & kBf16Bit) != 0;
        lo = p % kLine;
        base = reinterpret_cast<const char*>(p - lo);
        hi = lo + (n & ~kBf16Bit) * (bf16 ? 2 : 4);
    }
    // Byte offset of the current tile from `base`; moves to its tensor.
    __device__ __forceinline__ uint64_t offset() {
        if (tile >= a->first_tile[t + 1]) {
            do ++t; while (tile >= a->first_tile[t + 1]);
            enter();
        }
        return static_cast<uint64_t>(tile - a->first_tile[t]) * kTileBytes;
    }
};

template <bool BF16>
__device__ __forceinline__ void add_squares(const u32x4& x, double (&acc)[2]) {
#pragma unroll
    for (int e = 0; e < (BF16 ? 8 : 4); ++e) acc[e & 1] = square_to(acc[e & 1], rr::elem<BF16>(x, e));
}

// The squares of tile `at` of the tensor the walk is in.
template <bool BF16>
__device__ __forceinline__ void tile_squares(const char* base, uint64_t at, uint64_t lo, uint64_t hi,
                                             double (&acc)[2]) {
    constexpr uint32_t ES = BF16 ? 2 : 4;
    if (at >= lo && at + kTileBytes <= hi) {
        u32x4 x[kVecPerLane];
#pragma unroll
        for (int u = 0; u < kVecPerLane; ++u) x[u] = gv::load4(base + at + (u * kBlock + threadIdx.x) * 16u);
#pragma unroll
        for (int u = 0; u < kVecPerLane; ++u) add_squares<BF16>(x[u], acc);
        return;
    }
    // A tensor's first or last tile: whole vectors where they fit.
    for (int u = 0; u < kVecPerLane; ++u) {
        const uint64_t o = at + (u * kBlock + threadIdx.x) * 16u;
        if (o >= lo && o + 16 <= hi) {
            add_squares<BF16>(gv::load4(base + o), acc);
        } else {
            for (uint64_t e = o < lo ? lo : o; e < o + 16 && e < hi; e += ES)
                acc[0] = square_to(acc[0], gv::load_elem<BF16>(base + e));
        }
    }
}

__global__ __launch_bounds__(kBlock) void square_sum_kernel(NormArgs) {
    const auto a = (Konst<NormArgs>)(__builtin_amdgcn_kernarg_segment_ptr());
    double acc[2] = {0.0, 0.0};
    for (Walk<NormArgs> w(a); w.tile < w.last; ++w.tile) {
        const uint64_t at = w.offset();
        if (w.bf16) {
            tile_squares<true>(w.base, at, w.lo, w.hi, acc);
        } else {
            tile_squares<false>(w.base, at, w.lo, w.hi, acc);
        }
    }
    const double s = gv::block_sum<kBlock>(acc[0] + acc[1]);
    if (threadIdx.x == 0) {
        double* p = a->partials + blockIdx.x;
        *p = a->add ? *p + s : s;
    }
}

// Sum of count partials, the same in every lane of the workgroup.
__device__ __forceinline__ double sum_partials(const double* p, int64_t count) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kBlock) s += p[i];
    return gv::block_sum<kBlock>(s);
}

__global__ __launch_bounds__(kBlock) void norm_kernel(const double* partials, int64_t count, float* norm) {
    const double s = sum_partials(partials, count);
    if (threadIdx.x == 0) *norm = static_cast<float>(__builtin_sqrt(s));
}

// Partial b of gridDim.x: the sum of the b-th equal run of `count`.
__global__ __launch_bounds__(kBlock) void fold_kernel(const double* partials, int64_t count, double* to) {
    const int64_t lo = count * blockIdx.x / gridDim.x;
    const int64_t hi = count * (blockIdx.x + 1) / gridDim.x;
    const double s = sum_partials(partials + lo, hi - lo);
    if (threadIdx.x == 0) to[blockIdx.x] = s;
}

// x * c; a bf16 product is the float32 product rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ u32x4 scaled(const u32x4& x, float c) {
    u32x4 y;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (BF16) {
            y[k] = rr::bf16_bits(rr::elem<true>(x, 2 * k) * c) | (rr::bf16_bits(rr::elem<true>(x, 2 * k + 1) * c) << 16);
        } else {
            y[k] = __float_as_uint(__uint_as_float(x[k]) * c);
        }
    }
    return y;
}

template <bool BF16>
__device__ __forceinline__ void tile_scaled(const char* base, char* out, uint64_t at, uint64_t lo, uint64_t hi,
                                            float c) {
    constexpr uint32_t ES = BF16 ? 2 : 4;
    if (at >= lo && at + kTileBytes <= hi) {
        u32x4 x[kVecPerLane];
#pragma unroll
        for (int u = 0; u < kVecPerLane; ++u) x[u] = gv::load4(base + at + (u * kBlock + threadIdx.x) * 16u);
#pragma unroll
        for (int u = 0; u < kVecPerLane; ++u)
            gv::store4_nt(out + at + (u * kBlock + threadIdx.x) * 16u, scaled<BF16>(x[u], c));
        return;
    }
    for (int u = 0; u < kVecPerLane; ++u) {
        const uint64_t o = at + (u * kBlock + threadIdx.x) * 16u;
        if (o >= lo && o + 16 <= hi) {
            gv::store4_nt(out + o, scaled<BF16>(gv::load4(base + o), c));
        } else {
            for (uint64_t e = o < lo ? lo : o; e < o + 16 && e < hi; e += ES)
                gv::store_elem<BF16>(out + e, gv::load_elem<BF16>(base + e) * c);
        }
    }
}

__global__ __launch_bounds__(kBlock) void clip_kernel(ClipArgs) {
    const auto a = (Konst<ClipArgs>)(__builtin_amdgcn_kernarg_segment_ptr());
    float norm;
    if (a->n_partials > 0) {
        norm = static_cast<float>(__builtin_sqrt(sum_partials(a->partials, a->n_partials)));
        if (a->write_norm && blockIdx.x == 0 && threadIdx.x == 0) *a->norm = norm;
    } else {
        norm = *a->norm;
    }
    const float c = gv::clip_factor(norm, a->max_norm);
    if (a->in_place && c == 1.0f) return;   // what is there is the result
    for (Walk<ClipArgs> w(a); w.tile < w.last; ++w.tile) {
        const uint64_t at = w.offset();
        char* const out = a->out[w.t] - w.lo;
        if (w.bf16) {
            tile_scaled<true>(w.base, out, at, w.lo, w.hi, c);
        } else {
            tile_scaled<false>(w.base, out, at, w.lo, w.hi, c);
        }
    }
}

// Puts tensors from `t` on into one launch's arguments until they are full;
// returns the next tensor.  Empty tensors take no tile and no place.
template <class A, int CAP>
int32_t fill_set(const NormLaunch& l, int32_t t, A& a, bool out) {
    int64_t tiles = 0;
    a.n = 0;
    a.in_place = 1;
    for (; t < l.n_tensors && a.n < CAP; ++t) {
        if (l.numels[t] == 0) continue;
        const int64_t es = l.dtypes[t] == DDP_BF16 ? 2 : 4;
        const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(l.in[t]) % kLine);
        const int64_t need = (lead + l.numels[t] * es + kTileBytes - 1) / kTileBytes;
        if (tiles + need > kMaxTiles) break;
        a.in[a.n] = static_cast<const char*>(l.in[t]);
        if (out) {
            a.out[a.n] = static_cast<char*>(l.out[t]);
            if (l.out[t] != l.in[t]) a.in_place = 0;
        }
        a.numel[a.n] = static_cast<uint64_t>(l.numels[t]) | (es == 2 ? kBf16Bit : 0);
        a.first_tile[a.n] = static_cast<uint32_t>(tiles);
        tiles += need;
        ++a.n;
    }
    a.first_tile[a.n] = static_cast<uint32_t>(tiles);
    return t;
}

}  // namespace

int launch_square_sums(const NormLaunch& l, int* n_partials, const char** msg) {
    NormArgs a;
    *n_partials = 0;
    for (int32_t t = 0; t < l.n_tensors;) {
        t = fill_set<NormArgs, kNormCap>(l, t, a, false);
        if (a.n == 0) continue;
        // Every launch has as many workgroups as the first, so that each adds
        // to a partial that the first one wrote.
        a.add = *n_partials > 0;
        if (!a.add)
            *n_partials = t < l.n_tensors ? kNormPartials : static_cast<int>(std::min<uint32_t>(a.first_tile[a.n], kNormPartials));
        const int blocks = *n_partials;
        a.partials = l.partials;
        a.norm = nullptr;
        a.max_norm = 0.0f;
        a.n_partials = 0;
        a.write_norm = 0;
        void* args[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&square_sum_kernel), dim3(blocks),
                                             dim3(kBlock), args, 0, static_cast<hipStream_t>(l.stream));
        if (e != hipSuccess) {
            *msg = "hipLaunchKernel(square_sum)";
            return static_cast<int>(e);
        }
    }
    return 0;
}

int launch_norm_of(const double* partials, int64_t count, double* fold, float* norm, void* stream,
                   const char** msg) {
    // One workgroup adds 16,384 partials in about the time of a launch;
    // beyond that kNormFold of them go first.
    if (count > kNormFoldOver) {
        void* args[] = {&partials, &count, &fold};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&fold_kernel), dim3(kNormFold), dim3(kBlock),
                                             args, 0, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) {
            *msg = "hipLaunchKernel(fold)";
            return static_cast<int>(e);
        }
        partials = fold;
        count = kNormFold;
    }
    void* args[] = {&partials, &count, &norm};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&norm_kernel), dim3(1), dim3(kBlock), args, 0,
                                         static_cast<hipStream_t>(stream));
    if (e != hipSuccess) {
        *msg = "hipLaunchKernel(norm)";
        return static_cast<int>(e);
    }
    return 0;
}

int launch_clip(const NormLaunch& l, int n_partials, const char** msg) {
    ClipArgs a;
    bool first = true;
    for (int32_t t = 0; t < l.n_tensors;) {
        t = fill_set<ClipArgs, kClipCap>(l, t, a, true);
        if (a.n == 0) continue;
        const int grid = static_cast<int>(std::min<uint32_t>(a.first_tile[a.n], kNormPartials));
        a.partials = l.partials;
        a.n_partials = n_partials;
        a.norm = l.norm;
        a.max_norm = l.max_norm;
        a.write_norm = first;
        a.add = 0;
        first = false;
        void* args[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&clip_kernel), dim3(grid), dim3(kBlock),
                                             args, 0, static_cast<hipStream_t>(l.stream));
        if (e != hipSuccess) {
            *msg = "hipLaunchKernel(clip)";
            return static_cast<int>(e);
        }
    }
    return 0;
}

}  // namespace ddp

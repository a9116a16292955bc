// grad_norm.hip -- the global 2-norm of many gradient tensors and their
// clipping, for gfx950.
//
//     N = sqrt(sum over tensors and elements of g^2)
//     g <- g * min(1, max_norm / (N + 1e-6))
//
// Numbers.  The square of a float32 (or bf16) value is exact in float64 (24
// + 24 bits of 53) and neither overflows nor underflows there, so squares
// and sums are float64 throughout and the norm is rounded to float32 once.
// The sums' order is fixed by the tensors' sizes and starts: every wave or
// workgroup sums tiles of its own and leaves one partial, and the partials are
// added in order.  No atomics: the same tensors give the same bits every time.
//
// Layout.  A tile is a piece of one tensor that starts on a 128-byte line: the
// first tile of a tensor that starts inside a line is short by that much, so
// that a wave's accesses cover whole lines for any start.  The tensors'
// addresses and sizes travel in the kernel arguments (checked on the host,
// nothing on the device that could go stale); more tensors than one launch's
// arguments hold go out as several launches, the later ones adding to the
// partials of the earlier.
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

constexpr uint32_t kLine = 128;
constexpr uint32_t kVecPerLane = 4;                        // 16-byte vectors per lane and tile
constexpr uint32_t tile_bytes(int block) { return static_cast<uint32_t>(block) * kVecPerLane * 16u; }

// The norm: workgroups of 256 lanes, 16 KiB tiles, kNormPartials workgroups.
constexpr int kNormBlock = 256;
// The scaling: one-wave workgroups, 4 KiB tiles, one each.
constexpr int kClipBlock = 64;
// Both for few small tensors: one workgroup whose waves take 4 KiB tiles.
constexpr int kSmallBlock = 1024;
// The partials' sum.
constexpr int kSumBlock = 1024;

// The tensors of one launch.  numel's top bit says bf16.
template <int CAP, bool OUT>
struct SetArgs {
    static constexpr int kCap = CAP;
    static constexpr bool kOut = OUT;
    const char* in[CAP];
    char* out[OUT ? CAP : 1];
    uint64_t numel[CAP];
    uint32_t first_tile[CAP];
    int32_t n;                      // tensors, 1 .. CAP
    uint32_t tiles;                 // of all tensors
    int32_t add;                    // norm: add to the partials already there
    int32_t in_place;               // clip: every output is its input
    double* partials;
    float* norm;
    float max_norm;
};
constexpr uint64_t kBf16Bit = uint64_t(1) << 63;
typedef SetArgs<380, false> NormArgs;
typedef SetArgs<272, true> ClipArgs;
typedef SetArgs<kSmallTensors, true> SmallArgs;
static_assert(sizeof(NormArgs) <= 7800 && sizeof(ClipArgs) <= 7800,
              "kernel arguments must stay under the 8,000 bytes measured to pass");

template <class A>
using Konst = const __attribute__((address_space(4))) A*;
template <class A>
__device__ __forceinline__ Konst<A> args() {
    return (Konst<A>)(__builtin_amdgcn_kernarg_segment_ptr());
}

// The tensor a tile lies in.  All uniform.
struct Piece {
    const char* base;   // the tensor's start, down to a line
    uint64_t lo, hi;    // its bytes [lo, hi) from there
    uint64_t at;        // the tile's first byte from there
    bool bf16;
};
template <class A>
__device__ __forceinline__ Piece piece_of(Konst<A> a, int t, uint32_t tile, uint32_t bytes) {
    Piece p;
    const uint64_t in = reinterpret_cast<uint64_t>(a->in[t]);
    const uint64_t n = a->numel[t];
    p.bf16 = (n & kBf16Bit) != 0;
    p.lo = in % kLine;
    p.base = reinterpret_cast<const char*>(in - p.lo);
    p.hi = p.lo + (n & ~kBf16Bit) * (p.bf16 ? 2 : 4);
    p.at = static_cast<uint64_t>(tile - a->first_tile[t]) * bytes;
    return p;
}

// The tensor holding a tile: the last whose first tile is not past it.  For a
// workgroup that looks up one tile: a binary search with scalar loads.
template <class A>
__device__ __forceinline__ int tensor_at(Konst<A> a, uint32_t tile) {
    int lo = 0;
    for (int hi = a->n - 1; lo < hi;) {
        const int mid = (lo + hi + 1) >> 1;
        if (a->first_tile[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// For one that walks over many: every lane keeps some of the first tiles,
// and the tensor is the count of those not past the tile (a few compares and
// bit counts, no memory).
template <class A>
struct Finder {
    static constexpr int kRegs = (A::kCap + 63) / 64;
    uint32_t first[kRegs];

    __device__ __forceinline__ explicit Finder(Konst<A> a) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < kRegs; ++j) first[j] = j * 64 + lane < a->n ? a->first_tile[j * 64 + lane] : 0xffffffffu;
    }
    __device__ __forceinline__ int operator()(uint32_t tile) const {
        int t = -1;
#pragma unroll
        for (int j = 0; j < kRegs; ++j) t += __popcll(__ballot(first[j] <= tile));
        return t;
    }
};

template <bool BF16>
__device__ __forceinline__ void add_squares(const u32x4& x, double (&acc)[2]) {
#pragma unroll
    for (int e = 0; e < (BF16 ? 8 : 4); ++e) acc[e & 1] = square_to(acc[e & 1], rr::elem<BF16>(x, e));
}

// The squares of a tile, by BLOCK lanes of which this is `lane`.
template <int BLOCK, bool BF16>
__device__ __forceinline__ void tile_squares(const Piece& p, uint32_t lane, double (&acc)[2]) {
    constexpr uint32_t ES = BF16 ? 2 : 4;
    if (p.at >= p.lo && p.at + tile_bytes(BLOCK) <= p.hi) {
        u32x4 x[kVecPerLane];
#pragma unroll
        for (uint32_t u = 0; u < kVecPerLane; ++u) x[u] = gv::load4_nt(p.base + p.at + (u * BLOCK + lane) * 16u);
#pragma unroll
        for (uint32_t u = 0; u < kVecPerLane; ++u) add_squares<BF16>(x[u], acc);
        return;
    }
    // A tensor's first or last tile: whole vectors where they fit.
    for (uint32_t u = 0; u < kVecPerLane; ++u) {
        const uint64_t o = p.at + (u * BLOCK + lane) * 16u;
        if (o >= p.lo && o + 16 <= p.hi) {
            add_squares<BF16>(gv::load4(p.base + o), acc);
        } else {
            for (uint64_t e = o < p.lo ? p.lo : o; e < o + 16 && e < p.hi; e += ES)
                acc[0] = square_to(acc[0], gv::load_elem<BF16>(p.base + e));
        }
    }
}

template <int BLOCK>
__device__ __forceinline__ void tile_squares(const Piece& p, uint32_t lane, double (&acc)[2]) {
    if (p.bf16) {
        tile_squares<BLOCK, true>(p, lane, acc);
    } else {
        tile_squares<BLOCK, false>(p, lane, acc);
    }
}

__global__ __launch_bounds__(kNormBlock) void square_sum_kernel(NormArgs) {
    const Konst<NormArgs> a = args<NormArgs>();
    const Finder<NormArgs> find(a);
    const uint32_t tiles = a->tiles;
    double acc[2] = {0.0, 0.0};
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x)
        tile_squares<kNormBlock>(piece_of(a, find(tile), tile, tile_bytes(kNormBlock)), threadIdx.x, acc);
    const double s = gv::block_sum<kNormBlock>(acc[0] + acc[1]);
    if (threadIdx.x == 0) {
        double* p = a->partials + blockIdx.x;
        *p = a->add ? *p + s : s;
    }
}

// Sum of count partials, the same in every lane of the workgroup.
__device__ __forceinline__ double sum_partials(const double* p, int64_t count) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kSumBlock) s += p[i];
    return gv::block_sum<kSumBlock>(s);
}

__global__ __launch_bounds__(kSumBlock) void norm_kernel(const double* partials, int64_t count, float* norm) {
    const double s = sum_partials(partials, count);
    if (threadIdx.x == 0) *norm = static_cast<float>(__builtin_sqrt(s));
}

// The same for many partials: workgroup b sums the b-th equal run into
// fold[b], and the last one to finish adds those, in order.  fold[gridDim.x] is
// the count of finished ones, zero at the start.
__global__ __launch_bounds__(kSumBlock) void fold_kernel(const double* partials, int64_t count, double* fold,
                                                          float* norm) {
    const int64_t lo = count * blockIdx.x / gridDim.x;
    const int64_t hi = count * (blockIdx.x + 1) / gridDim.x;
    const double s = sum_partials(partials + lo, hi - lo);
    __shared__ uint32_t done;
    if (threadIdx.x == 0) {
        __hip_atomic_store(fold + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        done = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(fold + gridDim.x), 1u, __ATOMIC_ACQ_REL,
                                      __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (done != gridDim.x - 1) return;
    // The barrier put every lane after the release of all workgroups' sums.
    double x = 0.0;
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += kSumBlock)
        x += __hip_atomic_load(fold + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const double total = gv::block_sum<kSumBlock>(x);
    if (threadIdx.x == 0) *norm = static_cast<float>(__builtin_sqrt(total));
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

template <int BLOCK, bool BF16>
__device__ __forceinline__ void tile_scaled(const Piece& p, char* out, uint32_t lane, float c) {
    constexpr uint32_t ES = BF16 ? 2 : 4;
    if (p.at >= p.lo && p.at + tile_bytes(BLOCK) <= p.hi) {
        u32x4 x[kVecPerLane];
#pragma unroll
        for (uint32_t u = 0; u < kVecPerLane; ++u) x[u] = gv::load4_nt(p.base + p.at + (u * BLOCK + lane) * 16u);
#pragma unroll
        for (uint32_t u = 0; u < kVecPerLane; ++u)
            gv::store4_nt(out + p.at + (u * BLOCK + lane) * 16u, scaled<BF16>(x[u], c));
        return;
    }
    for (uint32_t u = 0; u < kVecPerLane; ++u) {
        const uint64_t o = p.at + (u * BLOCK + lane) * 16u;
        if (o >= p.lo && o + 16 <= p.hi) {
            gv::store4_nt(out + o, scaled<BF16>(gv::load4(p.base + o), c));
        } else {
            for (uint64_t e = o < p.lo ? p.lo : o; e < o + 16 && e < p.hi; e += ES)
                gv::store_elem<BF16>(out + e, gv::load_elem<BF16>(p.base + e) * c);
        }
    }
}

// out: the output tensor's start.
template <int BLOCK>
__device__ __forceinline__ void tile_scaled(const Piece& p, char* out, uint32_t lane, float c) {
    if (p.bf16) {
        tile_scaled<BLOCK, true>(p, out - p.lo, lane, c);
    } else {
        tile_scaled<BLOCK, false>(p, out - p.lo, lane, c);
    }
}

__global__ __launch_bounds__(kClipBlock) void clip_kernel(ClipArgs) {
    const Konst<ClipArgs> a = args<ClipArgs>();
    const float c = gv::clip_factor(gv::load_uniform(a->norm), a->max_norm);
    if (a->in_place && c == 1.0f) return;   // what is there is the result
    const uint32_t tiles = a->tiles;
    // From the last tile back: what was read last is likeliest in cache.
    for (uint32_t back = blockIdx.x; back < tiles; back += gridDim.x) {
        const uint32_t tile = tiles - 1 - back;
        const int t = tensor_at(a, tile);
        tile_scaled<kClipBlock>(piece_of(a, t, tile, tile_bytes(kClipBlock)), a->out[t], threadIdx.x, c);
    }
}

// The norm, and with CLIP the scaling by it, in one workgroup.
template <bool CLIP>
__global__ __launch_bounds__(kSmallBlock) void small_kernel(SmallArgs) {
    constexpr int kWaves = kSmallBlock / 64;
    const Konst<SmallArgs> a = args<SmallArgs>();
    const Finder<SmallArgs> find(a);
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tiles = a->tiles;
    double acc[2] = {0.0, 0.0};
    for (uint32_t tile = wave; tile < tiles; tile += kWaves)
        tile_squares<64>(piece_of(a, find(tile), tile, tile_bytes(64)), lane, acc);
    const float norm = static_cast<float>(__builtin_sqrt(gv::block_sum<kSmallBlock>(acc[0] + acc[1])));
    if (threadIdx.x == 0) *a->norm = norm;
    if constexpr (CLIP) {
        const float c = gv::clip_factor(norm, a->max_norm);
        if (a->in_place && c == 1.0f) return;
        for (uint32_t tile = wave; tile < tiles; tile += kWaves) {
            const int t = find(tile);
            tile_scaled<64>(piece_of(a, t, tile, tile_bytes(64)), a->out[t], lane, c);
        }
    }
}

// Puts tensors from `t` on into one launch's arguments until they are full;
// returns the next tensor.  Empty tensors take no tile and no place.
template <class A>
int32_t fill_set(const NormLaunch& l, int32_t t, uint32_t bytes, A& a) {
    int64_t tiles = 0;
    a.n = 0;
    a.in_place = 1;
    for (; t < l.n_tensors && a.n < A::kCap; ++t) {
        if (l.numels[t] == 0) continue;
        const int64_t es = l.dtypes[t] == DDP_BF16 ? 2 : 4;
        const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(l.in[t]) % kLine);
        const int64_t need = (lead + l.numels[t] * es + bytes - 1) / bytes;
        if (tiles + need > kMaxTiles) break;
        a.in[a.n] = static_cast<const char*>(l.in[t]);
        if constexpr (A::kOut) {
            if (l.out != nullptr) {
                a.out[a.n] = static_cast<char*>(l.out[t]);
                if (l.out[t] != l.in[t]) a.in_place = 0;
            }
        }
        a.numel[a.n] = static_cast<uint64_t>(l.numels[t]) | (es == 2 ? kBf16Bit : 0);
        a.first_tile[a.n] = static_cast<uint32_t>(tiles);
        tiles += need;
        ++a.n;
    }
    a.tiles = static_cast<uint32_t>(tiles);
    a.add = 0;
    a.partials = l.partials;
    a.norm = l.norm;
    a.max_norm = l.max_norm;
    return t;
}

int launch(const void* fn, unsigned grid, int block, void* arguments, unsigned lds, void* stream, const char* what,
           const char** msg) {
    void* list[] = {arguments};
    const hipError_t e =
        hipLaunchKernel(fn, dim3(grid), dim3(block), list, lds, static_cast<hipStream_t>(stream));
    if (e == hipSuccess) return 0;
    *msg = what;
    return static_cast<int>(e);
}

// The norm of every tensor by the wide kernel and the sum of its partials.
int launch_wide_norm(const NormLaunch& l, const char** msg) {
    NormArgs a;
    int blocks = 0;
    for (int32_t t = 0; t < l.n_tensors;) {
        t = fill_set(l, t, tile_bytes(kNormBlock), a);
        if (a.n == 0) continue;
        // Every launch has as many workgroups as the first, so that each adds
        // to a partial that the first one wrote.
        a.add = blocks > 0;
        if (!a.add)
            blocks = t < l.n_tensors ? kNormPartials : static_cast<int>(std::min<uint32_t>(a.tiles, kNormPartials));
        if (const int e = launch(reinterpret_cast<const void*>(&square_sum_kernel), blocks, kNormBlock, &a, 0, l.stream,
                                 "hipLaunchKernel(square_sum)", msg))
            return e;
    }
    return launch_norm_of(l.partials, blocks, nullptr, l.norm, l.stream, msg);
}

}  // namespace

int launch_norm_of(const double* partials, int64_t count, double* fold, float* norm, void* stream,
                   const char** msg) {
    void* many[] = {&partials, &count, &fold, &norm};
    void* few[] = {&partials, &count, &norm};
    const bool folds = count > kNormFoldOver;
    const hipError_t e =
        hipLaunchKernel(folds ? reinterpret_cast<const void*>(&fold_kernel) : reinterpret_cast<const void*>(&norm_kernel),
                        dim3(folds ? kNormFold : 1), dim3(kSumBlock), folds ? many : few, 0,
                        static_cast<hipStream_t>(stream));
    if (e == hipSuccess) return 0;
    *msg = folds ? "hipLaunchKernel(fold)" : "hipLaunchKernel(norm)";
    return static_cast<int>(e);
}

bool norm_is_small(int32_t n_tensors, const int64_t* numels, const int32_t* dtypes, bool clip) {
    int64_t n = 0, bytes = 0;
    for (int32_t t = 0; t < n_tensors; ++t) {
        if (numels[t] == 0) continue;
        bytes += numels[t] * (dtypes[t] == DDP_BF16 ? 2 : 4);
        if (++n > kSmallTensors || bytes > (clip ? kSmallClipBytes : kSmallNormBytes)) return false;
    }
    return n > 0;
}

int launch_norm(const NormLaunch& l, const char** msg) {
    if (!norm_is_small(l.n_tensors, l.numels, l.dtypes, false)) return launch_wide_norm(l, msg);
    SmallArgs a;
    fill_set(l, 0, tile_bytes(64), a);
    return launch(reinterpret_cast<const void*>(&small_kernel<false>), 1, kSmallBlock, &a, 0, l.stream,
                  "hipLaunchKernel(small norm)", msg);
}

int launch_clip(const NormLaunch& l, const char** msg) {
    if (!l.norm_given) {
        if (norm_is_small(l.n_tensors, l.numels, l.dtypes, true)) {
            SmallArgs a;
            fill_set(l, 0, tile_bytes(64), a);
            return launch(reinterpret_cast<const void*>(&small_kernel<true>), 1, kSmallBlock, &a, 0, l.stream,
                          "hipLaunchKernel(small clip)", msg);
        }
        if (const int e = launch_wide_norm(l, msg)) return e;
    }
    ClipArgs a;
    for (int32_t t = 0; t < l.n_tensors;) {
        t = fill_set(l, t, tile_bytes(kClipBlock), a);
        if (a.n == 0) continue;
        const unsigned grid = std::min(a.tiles, kMaxWaveGrid);
        if (const int e = launch(reinterpret_cast<const void*>(&clip_kernel), grid, kClipBlock, &a,
                                 lds_reserve(kClipWgPerCu), l.stream, "hipLaunchKernel(clip)", msg))
            return e;
    }
    return 0;
}

}  // namespace ddp

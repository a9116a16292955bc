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
// writes it once, and all of them are needed before the first can be scaled: a
// set larger than the caches is read twice.  What carries each kernel:
//   * the norm: 1,024 workgroups of 256 lanes take every 1,024th tile of 16
//     KiB, four non-temporal 16-byte loads a lane in flight.  2.0B bf16
//     elements 590 us with the partials' sum, 6.85 TB/s; 86.6M 29 us.  With
//     ordinary loads 6.0 TB/s; a contiguous run of tiles per workgroup 7% slower;
//     2,048 workgroups 4%.  2,048 one-wave workgroups are 3% faster on the 2.0B
//     elements, but lose 5% on 86.6M and 3% on ragged sets.
//   * the scaling: one one-wave workgroup per 4 KiB tile, 12 of them on a CU.
//     300M float32 370 us, 6.5 TB/s; 2,048 workgroups of 256 walking over the
//     tiles 5.1 TB/s, two tiles a workgroup 6.3.  In place with c = 1 all of
//     them start only to end, 63 us for 300M and 106 for 507M, where one read
//     of the norm is needed: not looked into yet, as it may cost c < 1 some
//     of its rate.
//   * few small tensors: one launch of one workgroup for norm and scaling.
//     24 tensors of 1,000 float32: norm 2.7 us on the GPU against 4.0 for the
//     wide kernels and 3.1 less per call on the host, clip 3.9 against 7.6 and
//     6.7 less per call; at the limit of 64 tiles level on the GPU (clip 7.0
//     against 6.1 us), and still less per call.
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
// Both for few small tensors: one workgroup whose waves hold up to four 4 KiB
// tiles each.
constexpr int kSmallBlock = 1024;
constexpr int kSmallWaves = kSmallBlock / 64;
constexpr int kSmallPerWave = kSmallTiles / kSmallWaves;
// The partials' sum.
constexpr int kSumBlock = 1024;

// The pieces of one launch: a tensor, or up to kMaxPiece elements of one.
// count's top bit says bf16.
template <int CAP, bool OUT>
struct SetArgs {
    static constexpr int kCap = CAP;
    static constexpr bool kOut = OUT;
    const char* in[CAP];
    char* out[OUT ? CAP : 1];
    uint32_t count[CAP];
    uint32_t first_tile[CAP];
    int32_t n;                      // pieces, 1 .. CAP
    uint32_t tiles;                 // of all pieces
    int32_t add;                    // norm: add to the partials already there
    int32_t in_place;               // clip: every output is its input
    double* partials;
    float* norm;
    float max_norm;
};
constexpr uint32_t kBf16Bit = 1u << 31;
typedef SetArgs<490, false> NormArgs;
typedef SetArgs<326, true> ClipArgs;
static_assert(sizeof(NormArgs) <= kArgBytes && sizeof(ClipArgs) <= kArgBytes, "kernel arguments");

template <class A>
using Konst = const __attribute__((address_space(4))) A*;
template <class A>
__device__ __forceinline__ Konst<A> args() {
    return (Konst<A>)(__builtin_amdgcn_kernarg_segment_ptr());
}

// The piece a tile lies in, and where.  All uniform.  Elements count from the
// piece's start; the tile's first one, on a line, may lie before it.
struct Piece {
    const char* in;
    int32_t n;
    int32_t at;
    bool bf16;
};
template <class A>
__device__ __forceinline__ Piece piece_of(Konst<A> a, int t, uint32_t tile, uint32_t bytes) {
    Piece p;
    p.in = a->in[t];
    const uint32_t count = a->count[t];
    p.bf16 = (count & kBf16Bit) != 0;
    p.n = static_cast<int32_t>(count & ~kBf16Bit);
    const uint32_t es = p.bf16 ? 1 : 2;   // shift
    p.at = static_cast<int32_t>((tile - a->first_tile[t]) * (bytes >> es)) -
           static_cast<int32_t>((reinterpret_cast<uint64_t>(p.in) % kLine) >> es);
    return p;
}

// The piece holding a tile: the last whose first tile is not past it.  For a
// workgroup that looks up one tile: a binary search with scalar loads.
template <class A>
__device__ __forceinline__ int piece_at(Konst<A> a, uint32_t tile) {
    int lo = 0;
    for (int hi = a->n - 1; lo < hi;) {
        const int mid = (lo + hi + 1) >> 1;
        if (a->first_tile[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// For one that walks over many: every lane keeps some of the first tiles,
// and the piece is the count of those not past the tile (a few compares and
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

// Whether a tile of BLOCK lanes lies inside its piece.
template <int BLOCK, bool BF16>
__device__ __forceinline__ bool inside(const Piece& p) {
    return p.at >= 0 && p.at + static_cast<int32_t>(tile_bytes(BLOCK) / (BF16 ? 2 : 4)) <= p.n;
}

// The element of the piece at which vector u of a lane of the tile starts.
template <int BLOCK, bool BF16>
__device__ __forceinline__ int32_t vector_at(const Piece& p, uint32_t u, uint32_t lane) {
    return p.at + static_cast<int32_t>((u * BLOCK + lane) * (BF16 ? 8u : 4u));
}

// A lane's vectors of a tile; in a piece's first and last tile zeros in the
// places past its ends, where single elements are read after all whole
// vectors are on their way.
template <int BLOCK, bool BF16>
__device__ __forceinline__ void load_tile(const Piece& p, uint32_t lane, u32x4 (&x)[kVecPerLane]) {
    constexpr int VE = BF16 ? 8 : 4;
    constexpr int64_t ES = BF16 ? 2 : 4;
    if (inside<BLOCK, BF16>(p)) {
#pragma unroll
        for (uint32_t u = 0; u < kVecPerLane; ++u) x[u] = gv::load4_nt(p.in + static_cast<int64_t>(vector_at<BLOCK, BF16>(p, u, lane)) * ES);
        return;
    }
#pragma unroll
    for (uint32_t u = 0; u < kVecPerLane; ++u) {
        const int32_t k = vector_at<BLOCK, BF16>(p, u, lane);
        x[u] = u32x4{0u, 0u, 0u, 0u};
        if (k >= 0 && k + VE <= p.n) x[u] = gv::load4_nt(p.in + static_cast<int64_t>(k) * ES);
    }
#pragma unroll
    for (uint32_t u = 0; u < kVecPerLane; ++u) {
        const int32_t k = vector_at<BLOCK, BF16>(p, u, lane);
        if ((k < 0 && k + VE > 0) || (k < p.n && k + VE > p.n)) x[u] = gv::load_some<BF16, VE>(p.in, k, p.n);
    }
}

template <int BLOCK, bool BF16>
__device__ __forceinline__ void tile_squares(const Piece& p, uint32_t lane, double (&acc)[2]) {
    u32x4 x[kVecPerLane];
    load_tile<BLOCK, BF16>(p, lane, x);
#pragma unroll
    for (uint32_t u = 0; u < kVecPerLane; ++u) add_squares<BF16>(x[u], acc);
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

// out: the output piece's start.
template <int BLOCK, bool BF16>
__device__ __forceinline__ void tile_scaled(const Piece& p, char* out, uint32_t lane, float c) {
    constexpr int VE = BF16 ? 8 : 4;
    constexpr int64_t ES = BF16 ? 2 : 4;
    u32x4 x[kVecPerLane];
    load_tile<BLOCK, BF16>(p, lane, x);
    if (inside<BLOCK, BF16>(p)) {
#pragma unroll
        for (uint32_t u = 0; u < kVecPerLane; ++u)
            gv::store4_nt(out + static_cast<int64_t>(vector_at<BLOCK, BF16>(p, u, lane)) * ES, scaled<BF16>(x[u], c));
        return;
    }
#pragma unroll
    for (uint32_t u = 0; u < kVecPerLane; ++u) {
        const int32_t k = vector_at<BLOCK, BF16>(p, u, lane);
        const u32x4 y = scaled<BF16>(x[u], c);
        if (k >= 0 && k + VE <= p.n) {
            gv::store4_nt(out + static_cast<int64_t>(k) * ES, y);
        } else {
            gv::store_some<BF16, VE>(out, k, p.n, y);
        }
    }
}

template <int BLOCK>
__device__ __forceinline__ void tile_scaled(const Piece& p, char* out, uint32_t lane, float c) {
    if (p.bf16) {
        tile_scaled<BLOCK, true>(p, out, lane, c);
    } else {
        tile_scaled<BLOCK, false>(p, out, lane, c);
    }
}

__global__ __launch_bounds__(kClipBlock) void clip_kernel(ClipArgs) {
    const Konst<ClipArgs> a = args<ClipArgs>();
    const float c = gv::clip_factor(gv::load_uniform(a->norm), a->max_norm);
    if (a->in_place && c == 1.0f) return;   // what is there is the result
    const uint32_t tiles = a->tiles;
    // From the last tile back.  (From the first on measures the same within 1%:
    // 300M float32 368 us back, 366 on; 507M 621 and 621; 86.6M bf16 after their
    // own norm 86 and 86.)
    for (uint32_t back = blockIdx.x; back < tiles; back += gridDim.x) {
        const uint32_t tile = tiles - 1 - back;
        const int t = piece_at(a, tile);
        tile_scaled<kClipBlock>(piece_of(a, t, tile, tile_bytes(kClipBlock)), a->out[t], threadIdx.x, c);
    }
}

// ---- few small tensors ------------------------------------------------------
//
// One launch of one workgroup: latency counts, not bandwidth.  The host cuts
// the tensors into tiles, so that a wave reads where its tiles are with one
// round of scalar loads; all its data is then in flight at once, and stays in
// registers until the norm is known and it is scaled and stored.

struct SmallArgs {
    const char* in[kSmallTiles];
    char* out[kSmallTiles];
    uint32_t count[kSmallTiles];    // elements, the top bit says bf16; 0 past the last tile
    int32_t in_place;
    float* norm;
    float max_norm;
};

// A lane's part of a tile: the whole vectors, and for the first lanes one
// element each of the rest.
struct Part {
    u32x4 x[kVecPerLane];
    uint32_t e;
};

template <bool BF16>
__device__ __forceinline__ void load_part(const char* in, uint32_t n, uint32_t lane, Part& p) {
    constexpr uint32_t VE = BF16 ? 8 : 4;
    constexpr uint32_t ES = BF16 ? 2 : 4;
    const uint32_t vectors = n / VE;
#pragma unroll
    for (uint32_t u = 0; u < kVecPerLane; ++u) {
        p.x[u] = u32x4{0u, 0u, 0u, 0u};
        if (u * 64 + lane < vectors) p.x[u] = gv::load4(in + (u * 64 + lane) * 16u);
    }
    p.e = 0;
    const uint32_t k = vectors * VE + lane;
    if (k < n) {
        if constexpr (BF16) {
            p.e = *reinterpret_cast<const uint16_t*>(in + k * ES);
        } else {
            p.e = *reinterpret_cast<const uint32_t*>(in + k * ES);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void add_part(const Part& p, double (&acc)[2]) {
#pragma unroll
    for (uint32_t u = 0; u < kVecPerLane; ++u) add_squares<BF16>(p.x[u], acc);
    acc[0] = square_to(acc[0], __uint_as_float(BF16 ? p.e << 16 : p.e));
}

template <bool BF16>
__device__ __forceinline__ void store_part(char* out, uint32_t n, uint32_t lane, const Part& p, float c) {
    constexpr uint32_t VE = BF16 ? 8 : 4;
    constexpr uint32_t ES = BF16 ? 2 : 4;
    const uint32_t vectors = n / VE;
#pragma unroll
    for (uint32_t u = 0; u < kVecPerLane; ++u)
        if (u * 64 + lane < vectors) gv::store4_nt(out + (u * 64 + lane) * 16u, scaled<BF16>(p.x[u], c));
    const uint32_t k = vectors * VE + lane;
    if (k < n) {
        if constexpr (BF16) {
            *reinterpret_cast<uint16_t*>(out + k * ES) = static_cast<uint16_t>(rr::bf16_bits(__uint_as_float(p.e << 16) * c));
        } else {
            *reinterpret_cast<float*>(out + k * ES) = __uint_as_float(p.e) * c;
        }
    }
}

template <bool CLIP>
__global__ __launch_bounds__(kSmallBlock) void small_kernel(SmallArgs) {
    const Konst<SmallArgs> a = args<SmallArgs>();
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t count[kSmallPerWave];
    const char* in[kSmallPerWave];
#pragma unroll
    for (int j = 0; j < kSmallPerWave; ++j) {
        count[j] = a->count[wave + j * kSmallWaves];
        in[j] = a->in[wave + j * kSmallWaves];
    }
    Part part[kSmallPerWave];
#pragma unroll
    for (int j = 0; j < kSmallPerWave; ++j) {
        if (count[j] == 0) continue;
        if (count[j] & kBf16Bit) {
            load_part<true>(in[j], count[j] & ~kBf16Bit, lane, part[j]);
        } else {
            load_part<false>(in[j], count[j], lane, part[j]);
        }
    }
    double acc[2] = {0.0, 0.0};
#pragma unroll
    for (int j = 0; j < kSmallPerWave; ++j) {
        if (count[j] == 0) continue;
        if (count[j] & kBf16Bit) {
            add_part<true>(part[j], acc);
        } else {
            add_part<false>(part[j], acc);
        }
    }
    const float norm = static_cast<float>(__builtin_sqrt(gv::block_sum<kSmallBlock>(acc[0] + acc[1])));
    if (threadIdx.x == 0) *a->norm = norm;
    if constexpr (CLIP) {
        const float c = gv::clip_factor(norm, a->max_norm);
        if (a->in_place && c == 1.0f) return;
#pragma unroll
        for (int j = 0; j < kSmallPerWave; ++j) {
            if (count[j] == 0) continue;
            char* const out = a->out[wave + j * kSmallWaves];
            if (count[j] & kBf16Bit) {
                store_part<true>(out, count[j] & ~kBf16Bit, lane, part[j], c);
            } else {
                store_part<false>(out, count[j], lane, part[j], c);
            }
        }
    }
}

// The tiles of one tensor: each ends on a line of its input.
int64_t small_tiles(const void* in, int64_t bytes) {
    const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(in) % kLine);
    return (lead + bytes + tile_bytes(64) - 1) / tile_bytes(64);
}

int launch_small(const NormLaunch& l, bool clip, const char** msg) {
    SmallArgs a{};
    a.in_place = 1;
    a.norm = l.norm;
    a.max_norm = l.max_norm;
    int tile = 0;
    for (int32_t t = 0; t < l.n_tensors; ++t) {
        if (l.numels[t] == 0) continue;
        const bool bf16 = l.dtypes[t] == DDP_BF16;
        const int64_t bytes = l.numels[t] * (bf16 ? 2 : 4);
        const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(l.in[t]) % kLine);
        if (clip && l.out[t] != l.in[t]) a.in_place = 0;
        for (int64_t at = -lead; at < bytes; at += tile_bytes(64), ++tile) {
            const int64_t lo = std::max<int64_t>(at, 0);
            const int64_t hi = std::min<int64_t>(at + tile_bytes(64), bytes);
            a.in[tile] = static_cast<const char*>(l.in[t]) + lo;
            if (clip) a.out[tile] = static_cast<char*>(l.out[t]) + lo;
            a.count[tile] = static_cast<uint32_t>((hi - lo) / (bf16 ? 2 : 4)) | (bf16 ? kBf16Bit : 0u);
        }
    }
    void* list[] = {&a};
    const hipError_t e = hipLaunchKernel(
        clip ? reinterpret_cast<const void*>(&small_kernel<true>) : reinterpret_cast<const void*>(&small_kernel<false>),
        dim3(1), dim3(kSmallBlock), list, 0, static_cast<hipStream_t>(l.stream));
    if (e == hipSuccess) return 0;
    *msg = "hipLaunchKernel(small norm)";
    return static_cast<int>(e);
}

// Where in a list of tensors the next launch goes on.
struct Place {
    int32_t t;
    int64_t at;    // element of tensor t
};

// Puts the tensors from `from` on into one launch's arguments until they are
// full; false when nothing was left.  Empty tensors take no place.
template <class A>
bool fill_set(const NormLaunch& l, Place& from, uint32_t bytes, A& a) {
    int64_t tiles = 0;
    a.n = 0;
    a.in_place = 1;
    for (; from.t < l.n_tensors && a.n < A::kCap; ++from.t, from.at = 0) {
        const int64_t es = l.dtypes[from.t] == DDP_BF16 ? 2 : 4;
        for (; from.at < l.numels[from.t] && a.n < A::kCap; ++a.n) {
            const int64_t count = std::min(l.numels[from.t] - from.at, kMaxPiece);
            const char* in = static_cast<const char*>(l.in[from.t]) + from.at * es;
            const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(in) % kLine);
            a.in[a.n] = in;
            if constexpr (A::kOut) {
                a.out[a.n] = static_cast<char*>(l.out[from.t]) + from.at * es;
                if (a.out[a.n] != in) a.in_place = 0;
            }
            a.count[a.n] = static_cast<uint32_t>(count) | (es == 2 ? kBf16Bit : 0);
            a.first_tile[a.n] = static_cast<uint32_t>(tiles);
            tiles += (lead + count * es + bytes - 1) / bytes;
            from.at += count;
        }
        if (from.at < l.numels[from.t]) break;
    }
    a.tiles = static_cast<uint32_t>(tiles);
    a.add = 0;
    a.partials = l.partials;
    a.norm = l.norm;
    a.max_norm = l.max_norm;
    return a.n > 0;
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
    for (Place at = {0, 0}; fill_set(l, at, tile_bytes(kNormBlock), a);) {
        // Every launch has as many workgroups as the first, so that each adds
        // to a partial that the first one wrote.
        a.add = blocks > 0;
        if (!a.add)
            blocks = at.t < l.n_tensors ? kNormPartials : static_cast<int>(std::min<uint32_t>(a.tiles, kNormPartials));
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

bool norm_is_small(int32_t n_tensors, const int64_t* numels, const void* const* in, const int32_t* dtypes) {
    int64_t tiles = 0;
    for (int32_t t = 0; t < n_tensors && tiles <= kSmallTiles; ++t)
        if (numels[t] > 0) tiles += small_tiles(in[t], numels[t] * (dtypes[t] == DDP_BF16 ? 2 : 4));
    return tiles > 0 && tiles <= kSmallTiles;
}

int launch_norm(const NormLaunch& l, const char** msg) {
    return l.partials == nullptr ? launch_small(l, false, msg) : launch_wide_norm(l, msg);
}

int launch_clip(const NormLaunch& l, const char** msg) {
    if (!l.norm_given) {
        if (l.partials == nullptr) return launch_small(l, true, msg);
        if (const int e = launch_wide_norm(l, msg)) return e;
    }
    ClipArgs a;
    for (Place at = {0, 0}; fill_set(l, at, tile_bytes(kClipBlock), a);) {
        const unsigned grid = std::min(a.tiles, kMaxWaveGrid);
        if (const int e = launch(reinterpret_cast<const void*>(&clip_kernel), grid, kClipBlock, &a,
                                 lds_reserve(kClipWgPerCu), l.stream, "hipLaunchKernel(clip)", msg))
            return e;
    }
    return 0;
}

}  // namespace ddp

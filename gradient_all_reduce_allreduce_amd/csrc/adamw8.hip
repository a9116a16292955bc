// adamw8.hip -- one AdamW step on many tensors with the moments kept in 8
// bits, the gradient clipped on the way, and the moments read back, for gfx950.
//
// The step is adamw.hip's (adamw_math.h), in float32 on decoded moments; the
// new moments are rounded to 8 bits after the weights have used them.  A block
// is 32 consecutive elements of a tensor with two scale bytes, of m and of v.
//
//   m  sign, 4 bits of exponent, 3 of mantissa (up to 448), times
//      2^(s - 127); s the smallest, from 1, that holds the block's maximum.
//   v  5 bits of exponent, 3 of mantissa, no sign: code c times scale is
//      (1 + (c & 7) / 8) * 2^((c >> 3) - 31) * 2^(s - 127), at most 1.875 scales;
//      s the smallest, from 32, that holds the block's maximum, 0 for a block
//      of zeros.  No code is zero: beside the largest of the block even 0
//      stands for 2^-31 scales, so a first moment is never divided by eps alone
//      because its second one was rounded away.
//
// Rounding is at random, up with the probability of the part cut off.  Rounded
// to nearest, a moment stops where its change per step falls under half a step
// of its code: v, which moves by (1 - b2) of itself, at a sixteenth of its
// value for b2 = 0.999, and the weights' steps come out several times too long.
// At random, the expected moment is the exact one.  With one step's share of
// (1 - b2) and codes d apart (d = 1/16 .. 1/8 of the value) a stationary v has
// a relative standard deviation of about sqrt(d / 2), 20-25%, from the rounding,
// whatever b2; m, which moves by more than its code's step, about 8%.
//
// A block of m with an infinity or a NaN has s = 255 and is NaN as a whole from
// the next step on, one of v infinite.  A norm that is not finite leaves
// everything as it was.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "adamw_math.h"
#include "launch_mx.h"
#include "mx.h"

namespace ddp {
namespace {

using rr::u32x2;
using rr::u32x4;

constexpr uint32_t kTileElems = 256;
constexpr uint32_t kBlockElems = DDP_MX_BLOCK;
// Tensors (or pieces of them) per launch: as many as the arguments hold.
constexpr int kCap = 120;

struct Adam8Args {
    const char* g[kCap];
    char* w[kCap];
    char* m[kCap];
    char* v[kCap];
    char* s[kCap];
    char* p[kCap];
    uint32_t count[kCap];      // elements, up to kMaxPiece
    uint32_t first_tile[kCap];
    uint32_t tensor[kCap];     // which tensor of the call a piece belongs to,
    uint32_t piece[kCap];      // and which of its pieces it is
    int32_t n;
    uint32_t tiles;
    uint32_t seed;             // the seed's two halves mixed
    adamw::Scalars scalars;
};
static_assert(sizeof(Adam8Args) <= kArgBytes, "kernel arguments");
typedef const __attribute__((address_space(4))) Adam8Args* KAdam8;

// Random bits.  32 per element, from a key and the element's place in its
// piece: a multiplication by 2^32 over the golden ratio steps through all
// values, and one more round (the fraction of the root of 3) makes neighbours
// independent (joint frequencies of pairs at 19 distances from 1 to 10^6, over
// 200,000 keys, within 3.1 standard deviations).  A key is the seed, the
// step's number, the tensor's and the piece's, each through two rounds.
constexpr uint32_t kGolden = 0x9E3779B9u;
constexpr uint32_t kRoot3 = 0xBB67AE85u;
constexpr uint32_t kRoot5 = 0x3C6EF373u;

__host__ __device__ __forceinline__ uint32_t mix_word(uint32_t h, uint32_t word) {
    uint32_t x = (h ^ word) + kGolden;
    x ^= x >> 16;
    x *= kRoot3;
    x ^= x >> 15;
    x *= kRoot5;
    return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t random_bits(uint32_t x) {
    x ^= x >> 15;
    x *= kRoot3;
    return x ^ (x >> 16);
}

// What is added to a float32's bits below the 4 kept: 16 random bits and a
// half, so that neither side is favoured by the rest that they leave out.
__device__ __forceinline__ uint32_t low_bits(uint32_t r) { return ((r & 0xffffu) << 4) | 8u; }
__device__ __forceinline__ uint32_t high_bits(uint32_t r) { return ((r >> 12) & 0xffff0u) | 8u; }

__device__ __forceinline__ float decode_v(uint32_t code, float scale) {
    return __uint_as_float((code << 20) + (96u << 23)) * scale;
}

// The scale byte of m from the largest magnitude's bits: with that rounded up
// to 3 bits of mantissa, its exponent less 8, one more for 1.875, which has no
// code (it would be NaN's).
__device__ __forceinline__ uint32_t scale_m(uint32_t top) {
    const uint32_t e = ((((top + 0xfffffu) >> 20) + 1u) >> 3);
    return top < 0x7f800000u ? mx::larger(e, 9u) - 8u : 255u;
}
__device__ __forceinline__ uint32_t scale_v(uint32_t top) {
    const uint32_t e = (top + 0xfffffu) >> 23;
    if (top == 0u) return 0u;
    return e < 255u ? mx::larger(e, 32u) : 255u;
}

// up: 2^(127 - s), which brings the block's maximum to at most 448.
__device__ __forceinline__ uint32_t encode_m(float m, float up, uint32_t r) {
    const float x = __builtin_fabsf(m) * up;
    const uint32_t normal = ((__float_as_uint(x) + r) >> 20) - (120u << 3);
    const uint32_t small = (static_cast<uint32_t>(__builtin_fminf(x, 0x1p-6f) * 0x1p29f) + r) >> 20;   // steps of 2^-9
    return (x < 0x1p-6f ? small : normal) | ((__float_as_uint(m) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t encode_v(float v, uint32_t s, uint32_t r) {
    const int32_t c = static_cast<int32_t>((__float_as_uint(v) + r) >> 20) - (static_cast<int32_t>(s - 31u) << 3);
    return static_cast<uint32_t>(c < 0 ? 0 : c);
}

// Four bytes at any address, and those of them that lie in [0, n).
typedef uint32_t __attribute__((aligned(1))) u32_any;
typedef __attribute__((address_space(1))) const u32_any* GlobalIn1;
typedef __attribute__((address_space(1))) u32_any* GlobalOut1;
__device__ __forceinline__ uint32_t load_bytes(const char* p, int64_t i, int64_t n, bool whole) {
    if (whole) return *(GlobalIn1)(p + i);
    uint32_t x = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i + e < n) x |= static_cast<uint32_t>(static_cast<uint8_t>(p[i + e])) << (8 * e);
    return x;
}
__device__ __forceinline__ void store_bytes(char* p, int64_t i, int64_t n, bool whole, uint32_t x) {
    if (whole) {
        *(GlobalOut1)(p + i) = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i + e < n) p[i + e] = static_cast<char>(x >> (8 * e));
}

// The last piece that starts at or before the tile.
template <class A>
__device__ __forceinline__ int piece_of(A a, uint32_t tile) {
    int t = 0;
    for (int h = a->n - 1; t < h;) {
        const int mid = (t + h + 1) >> 1;
        if (a->first_tile[mid] <= tile) t = mid; else h = mid - 1;
    }
    return t;
}

// GB: bf16 gradients.  PM: the copy, 0 none, 1 float32, 2 bf16.
template <bool GB, int PM>
__global__ __launch_bounds__(mx::kWave) void adamw8_kernel(Adam8Args) {
    const KAdam8 a = (KAdam8)(__builtin_amdgcn_kernarg_segment_ptr());
    const uint32_t tiles = a->tiles;
    const adamw::KScalars k = (adamw::KScalars)(&a->scalars);
    const float norm = k->norm != nullptr ? gv::load_uniform(k->norm) : 0.0f;
    const int64_t step = k->step != nullptr ? gv::load_uniform(k->step) : k->host_step;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int t = piece_of(a, tile);
        const char* const g = a->g[t];
        char* const w = a->w[t];
        char* const m = a->m[t];
        char* const v = a->v[t];
        char* const s = a->s[t];
        char* const p = a->p[t];
        const int64_t n = a->count[t];
        const int64_t at = static_cast<int64_t>(tile - a->first_tile[t]) * kTileElems;
        const int64_t i = at + threadIdx.x * 4;
        const bool whole = at + kTileElems <= n || i + 4 <= n;
        const bool held = i / kBlockElems * kBlockElems < n;
        u32x4 gq, wq;
        if (whole) {
            if constexpr (GB) {
                const u32x2 h = gv::load2_nt(g + i * 2);
                gq = u32x4{h[0], h[1], 0u, 0u};
            } else {
                gq = gv::load4_nt(g + i * 4);
            }
            wq = gv::load4_nt(w + i * 4);
        } else {
            gq = gv::load_some<GB, 4>(g, i, n);
            wq = gv::load_some<false, 4>(w, i, n);
        }
        const uint32_t mq = load_bytes(m, i, n, whole);
        const uint32_t vq = load_bytes(v, i, n, whole);
        char* const sp = s + i / kBlockElems * 2;
        const uint32_t sq = held ? *reinterpret_cast<const uint16_t*>(sp) : 0u;
        adamw::Factors f;
        if (!adamw::factors(k, norm, step, f)) return;
        uint32_t key = mix_word(a->seed, static_cast<uint32_t>(step));
        key = mix_word(key, static_cast<uint32_t>(step >> 32));
        key = mix_word(mix_word(key, a->tensor[t]), a->piece[t]);
        const uint32_t x0 = key + static_cast<uint32_t>(i) * kGolden;

        const float ms = mx::scale_of(sq & 0xffu);
        const float vs = mx::scale_of(sq >> 8);
        const mx::f32x2 m01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(mq, ms, false);
        const mx::f32x2 m23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(mq, ms, true);
        float me[4] = {m01[0], m01[1], m23[0], m23[1]};
        float ve[4], wn[4];
        uint32_t mtop = 0, vtop = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ve[e] = decode_v((vq >> (8 * e)) & 0xffu, vs);
            wn[e] = __uint_as_float(wq[e]);
            adamw::adamw_element(rr::elem<GB>(gq, e), wn[e], me[e], ve[e], f);
            wq[e] = __float_as_uint(wn[e]);
            if (i + e < n) {
                mtop = mx::larger(mtop, __float_as_uint(me[e]) & 0x7fffffffu);
                vtop = mx::larger(vtop, __float_as_uint(ve[e]) & 0x7fffffffu);
            }
        }
        const uint32_t sm = scale_m(mx::max_of_8(mtop));
        const uint32_t sv = scale_v(mx::max_of_8(vtop));
        const float up = __uint_as_float((254u - (sm < 254u ? sm : 254u)) << 23);
        uint32_t mc = 0, vc = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t r = random_bits(x0 + e * kGolden);
            mc |= encode_m(me[e], up, low_bits(r)) << (8 * e);
            vc |= encode_v(ve[e], sv, high_bits(r)) << (8 * e);
        }
        if (sm == 255u) mc = 0x7f7f7f7fu;
        if (sv == 255u || sv == 0u) vc = 0u;
        store_bytes(m, i, n, whole, mc);
        store_bytes(v, i, n, whole, vc);
        if (held && (threadIdx.x & 7) == 0) *reinterpret_cast<uint16_t*>(sp) = static_cast<uint16_t>(sm | sv << 8);
        const u32x2 h = {rr::bf16_bits(wn[0]) | (rr::bf16_bits(wn[1]) << 16),
                         rr::bf16_bits(wn[2]) | (rr::bf16_bits(wn[3]) << 16)};
        if (whole) {
            gv::store4_nt(w + i * 4, wq);
            if constexpr (PM == 1) gv::store4_nt(p + i * 4, wq);
            if constexpr (PM == 2) gv::store2_nt(p + i * 2, h);
        } else {
            gv::store_some<false, 4>(w, i, n, wq);
            if constexpr (PM == 1) gv::store_some<false, 4>(p, i, n, wq);
            if constexpr (PM == 2) gv::store_some<true, 4>(p, i, n, u32x4{h[0], h[1], 0u, 0u});
        }
    }
}

const void* kernel_for(const AdamWLaunch& l) {
    const int pm = l.params == nullptr ? 0 : (l.param_bf16 ? 2 : 1);
    if (l.grad_bf16) {
        return pm == 0 ? reinterpret_cast<const void*>(&adamw8_kernel<true, 0>)
               : pm == 1 ? reinterpret_cast<const void*>(&adamw8_kernel<true, 1>)
                         : reinterpret_cast<const void*>(&adamw8_kernel<true, 2>);
    }
    return pm == 0 ? reinterpret_cast<const void*>(&adamw8_kernel<false, 0>)
           : pm == 1 ? reinterpret_cast<const void*>(&adamw8_kernel<false, 1>)
                     : reinterpret_cast<const void*>(&adamw8_kernel<false, 2>);
}

// The moments' values.
struct Read8Args {
    const char* m[kCap];
    const char* v[kCap];
    const char* s[kCap];
    char* m_out[kCap];
    char* v_out[kCap];
    uint32_t count[kCap];
    uint32_t first_tile[kCap];
    int32_t n;
    uint32_t tiles;
};
static_assert(sizeof(Read8Args) <= kArgBytes, "kernel arguments");
typedef const __attribute__((address_space(4))) Read8Args* KRead8;

template <bool BF16>
__global__ __launch_bounds__(mx::kWave) void adamw8_read_kernel(Read8Args) {
    const KRead8 a = (KRead8)(__builtin_amdgcn_kernarg_segment_ptr());
    const uint32_t tiles = a->tiles;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int t = piece_of(a, tile);
        const int64_t n = a->count[t];
        const int64_t at = static_cast<int64_t>(tile - a->first_tile[t]) * kMxTileElems;
        const int64_t i = at + threadIdx.x * 8;
        if (i >= n) continue;
        const bool whole = i + 8 <= n;
        const char* const sp = a->s[t] + i / kBlockElems * 2;
        const uint32_t sq = *reinterpret_cast<const uint16_t*>(sp);
        float m[8], v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t mq = load_bytes(a->m[t], i + 4 * h, n, whole);
            const uint32_t vq = load_bytes(a->v[t], i + 4 * h, n, whole);
            const mx::f32x2 m01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(mq, mx::scale_of(sq & 0xffu), false);
            const mx::f32x2 m23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(mq, mx::scale_of(sq & 0xffu), true);
            m[4 * h] = m01[0], m[4 * h + 1] = m01[1], m[4 * h + 2] = m23[0], m[4 * h + 3] = m23[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * h + e] = decode_v((vq >> (8 * e)) & 0xffu, mx::scale_of(sq >> 8));
        }
        mx::store_oct<BF16>(a->m_out[t], i, n, whole, mx::pack_oct<BF16>(m));
        mx::store_oct<BF16>(a->v_out[t], i, n, whole, mx::pack_oct<BF16>(v));
    }
}

int launch(const void* fn, void* args, uint32_t tiles, unsigned lds, void* stream, const char* what, const char** msg) {
    void* list[] = {args};
    const hipError_t e = hipLaunchKernel(fn, dim3(std::min(tiles, kMaxWaveGrid)), dim3(mx::kWave), list, lds,
                                         static_cast<hipStream_t>(stream));
    if (e == hipSuccess) return 0;
    *msg = what;
    return static_cast<int>(e);
}

}  // namespace

int launch_adamw8(const AdamW8Launch& l, const char** msg) {
    const AdamWLaunch& b = l.step;
    Adam8Args a;
    a.scalars = adamw::scalars_of(b);
    a.seed = mix_word(mix_word(0, static_cast<uint32_t>(l.seed)), static_cast<uint32_t>(l.seed >> 32));
    const void* fn = kernel_for(b);
    int64_t at = 0;   // element of tensor t that the next piece starts at
    for (int32_t t = 0; t < b.n_tensors;) {
        int64_t tiles = 0;
        for (a.n = 0; t < b.n_tensors && a.n < kCap;) {
            const int64_t count = std::min(b.numels[t] - at, kMaxPiece);
            if (count > 0) {
                a.g[a.n] = static_cast<const char*>(b.grads[t]) + at * (b.grad_bf16 ? 2 : 4);
                a.w[a.n] = reinterpret_cast<char*>(b.w[t] + at);
                a.m[a.n] = reinterpret_cast<char*>(l.m[t] + at);
                a.v[a.n] = reinterpret_cast<char*>(l.v[t] + at);
                a.s[a.n] = reinterpret_cast<char*>(l.scales[t] + at / kBlockElems * 2);
                a.p[a.n] = b.params != nullptr ? static_cast<char*>(b.params[t]) + at * (b.param_bf16 ? 2 : 4) : nullptr;
                a.count[a.n] = static_cast<uint32_t>(count);
                a.first_tile[a.n] = static_cast<uint32_t>(tiles);
                a.tensor[a.n] = static_cast<uint32_t>(t);
                a.piece[a.n] = static_cast<uint32_t>(at / kMaxPiece);
                tiles += (count + kTileElems - 1) / kTileElems;
                at += count;
                ++a.n;
            }
            if (at >= b.numels[t]) {
                ++t;
                at = 0;
            }
        }
        if (a.n == 0) continue;
        a.tiles = static_cast<uint32_t>(tiles);
        if (const int e = launch(fn, &a, a.tiles, 0, b.stream, "hipLaunchKernel(adamw8)", msg)) return e;
    }
    return 0;
}

int launch_adamw8_read(const Moments8Read& l, const char** msg) {
    Read8Args a;
    const void* fn = l.out_bf16 ? reinterpret_cast<const void*>(&adamw8_read_kernel<true>)
                                : reinterpret_cast<const void*>(&adamw8_read_kernel<false>);
    const int64_t es = l.out_bf16 ? 2 : 4;
    int64_t at = 0;
    for (int32_t t = 0; t < l.n_tensors;) {
        int64_t tiles = 0;
        for (a.n = 0; t < l.n_tensors && a.n < kCap;) {
            const int64_t count = std::min(l.numels[t] - at, kMaxPiece);
            if (count > 0) {
                a.m[a.n] = reinterpret_cast<const char*>(l.m[t] + at);
                a.v[a.n] = reinterpret_cast<const char*>(l.v[t] + at);
                a.s[a.n] = reinterpret_cast<const char*>(l.scales[t] + at / kBlockElems * 2);
                a.m_out[a.n] = static_cast<char*>(l.m_out[t]) + at * es;
                a.v_out[a.n] = static_cast<char*>(l.v_out[t]) + at * es;
                a.count[a.n] = static_cast<uint32_t>(count);
                a.first_tile[a.n] = static_cast<uint32_t>(tiles);
                tiles += mx_tiles(count);
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
        if (const int e = launch(fn, &a, a.tiles, 0, l.stream, "hipLaunchKernel(adamw8_read)", msg)) return e;
    }
    return 0;
}

}  // namespace ddp

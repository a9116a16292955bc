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
// At random, the expected moment is the exact one.  Codes are d = 1/16 to 1/8 of
// the value apart, and a v whose steps are smaller than that varies about the
// exact one by sqrt(d / 2) of it, whatever b2 (18% with normal gradients and b2 =
// 0.99, 20% with 0.999, no offset); m, whose steps are larger, by 9% of its own
// root mean square.
//
// A block of m with an infinity or a NaN, of whatever sign and payload, has s = 255
// and is NaN as a whole from the next step on, one of v infinite.  A norm that is
// not finite leaves everything as it was.
//
// Bound by HBM: 16.1 bytes an element with bf16 gradient and copy (32-bit moments:
// 28) against 64 instructions, 11 of them a wave's own.  86.6M elements, bf16
// gradient and copy: 221 us, 6.3 TB/s, with the count on the GPU 222; float32
// gradient without copy 221, one element off a line 236.  Read back as bf16 82 us,
// 6.4 TB/s, as float32 130, 6.7.
//
// Layout: a workgroup of 4 waves takes a tile of 2,048 elements, a wave two spans
// of 256, all loads of both first; a lane has 4 consecutive elements, 16 bytes of
// the weights, and 8 lanes a block.  Blocks count from the tensor's first element,
// so tiles do too, wherever that lies in a line.  One span a wave took 267 us, 279
// with the count on the GPU, when two took 231 and 237; four 226 when two took 221.
// A short call's waves take one: 1,000 elements 3.9 us instead of 5.0, 1M 5.4 and
// 5.6, 2M 9.0 and 8.2.  By workgroups per CU 0 (full), 2, 3, 4, 5, 6, 8: 228 261 227
// 221 227 224 226 us.  Addresses and sizes travel in the kernel arguments, as in
// adamw.hip, 161 tensors a launch (139 with copies of the weights).
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

// Workgroups of 4 waves; a wave takes kSpans spans (one in a short launch) of 256
// consecutive elements, a lane 4 of each, 8 lanes a block.
constexpr unsigned kLanes = 256;
constexpr uint32_t kSpan = 256;
constexpr int kSpans = 2;
constexpr uint32_t kBlockElems = DDP_MX_BLOCK;
constexpr uint32_t kMaxGrid = 1u << 23;
constexpr int rows_for(int cap) { return (cap + 15) / 16 * 16; }
// Consecutive tensors of a call, as many as the arguments hold (PARAMS: with
// their copies), empty ones among them; or one piece of a tensor that is longer
// than kMaxPiece.
template <bool PARAMS>
struct Adam8Args {
    static constexpr int kCap = PARAMS ? 139 : 161, kRows = rows_for(kCap);
    const char* g[kCap];
    char* w[kCap];
    char* m[kCap];
    char* v[kCap];
    char* s[kCap];
    char* p[PARAMS ? kCap : 1];
    uint32_t count[kCap];      // elements
    uint32_t first_tile[kRows];    // behind the last tensor none that a tile can have
    int32_t n;
    uint32_t tiles;
    uint32_t tensor;           // the first one's number in the call
    uint32_t piece;            // and which of its pieces it is
    uint32_t seed;             // the seed's two halves mixed
    adamw::Scalars scalars;
};
static_assert(sizeof(Adam8Args<false>) <= kArgBytes && sizeof(Adam8Args<true>) <= kArgBytes, "kernel arguments");

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
// The same of v; a NaN, which lies above infinity and may have a sign, counts as
// infinity, so that the sum stays within 32 bits.
__device__ __forceinline__ uint32_t scale_v(uint32_t top) {
    const uint32_t e = ((top < 0x7f800000u ? top : 0x7f800000u) + 0xfffffu) >> 23;
    if (top == 0u) return 0u;
    return e < 255u ? mx::larger(e, 32u) : 255u;
}

// A moment's code is what a float32's exponent and top 3 bits of mantissa are
// once its exponent starts where the code's does; the 20 bits below are the part
// cut off, and 16 random bits and a half (neither side is favoured by the rest
// that they leave out), added to them, carry into the code with its probability.
// m, in scales (up = 2^(127 - s)) and times 2^-120, is subnormal just where its
// code is: the code with the sign in front lies in the top byte.
__device__ __forceinline__ uint32_t encode_m(float m, float up, uint32_t r) {
#pragma clang fp contract(off)
    const float x = __builtin_fabsf(m) * up * 0x1p-120f;
    const uint32_t t = __float_as_uint(x) + ((r & 0xffffu) << 4) + 8u;
    return (__float_as_uint(m) & 0x80000000u) | ((t << 4) & 0x7fffffffu);
}
// v less what its exponent starts at (`from`, and the half); below that code 0.
__device__ __forceinline__ uint32_t encode_v(float v, uint32_t from, uint32_t r) {
    const int32_t t = static_cast<int32_t>(__float_as_uint(v) + ((r >> 16) << 4) + from);
    return static_cast<uint32_t>(t < 0 ? 0 : t) << 4;
}
// The top bytes of four words.
__device__ __forceinline__ uint32_t top_bytes(const uint32_t (&x)[4]) {
    const uint32_t lo = __builtin_amdgcn_perm(x[1], x[0], 0x0c0c0703u);
    return __builtin_amdgcn_perm(x[3], x[2], 0x07030c0cu) | lo;
}

// The weights' step, the root and the quotient by the hardware's instructions,
// within 1 ulp each: beside moments of 3 bits of mantissa a correctly rounded one
// says nothing more (the largest error of float32 weights grows by some 2%).  Both
// rounded correctly cost what bf16 gradients leave of the instructions' time: 86.6M
// elements with a bf16 copy 231 us instead of 223, with the count on the GPU too 238
// instead of 221, without a copy 208 instead of 193; float32 gradients 219 and 218.
// A second moment below 2^-126, which these instructions take for zero, counts as
// that.
__device__ __forceinline__ float step_weight(float w, float m, float v, const adamw::Factors& f) {
#pragma clang fp contract(off)
    const float least = __uint_as_float(mx::larger(__float_as_uint(v), 1u << 23));
    const float d = __builtin_amdgcn_sqrtf(least) * f.root2 + f.eps;
    const float q = m * __builtin_amdgcn_rcpf(d);
    const float w0 = w * f.decay;
    const float s = f.step_size * q;
    return w0 - s;
}

// Four bytes at any address, those of them that lie in [0, n) unless WHOLE.
typedef uint32_t __attribute__((aligned(1))) u32_any;
typedef __attribute__((address_space(1))) const u32_any* GlobalIn1;
typedef __attribute__((address_space(1))) u32_any* GlobalOut1;
template <bool WHOLE>
__device__ __forceinline__ uint32_t load_bytes(const char* p, int64_t i, int64_t n) {
    if constexpr (WHOLE) return __builtin_nontemporal_load((GlobalIn1)(p + i));
    uint32_t x = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i + e < n) x |= static_cast<uint32_t>(static_cast<uint8_t>(p[i + e])) << (8 * e);
    return x;
}
template <bool WHOLE>
__device__ __forceinline__ void store_bytes(char* p, int64_t i, int64_t n, uint32_t x) {
    if constexpr (WHOLE) {
        __builtin_nontemporal_store(x, (GlobalOut1)(p + i));
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i + e < n) p[i + e] = static_cast<char>(x >> (8 * e));
}

// The last tensor that starts at or before the tile: counted among every 16th,
// then among the 16 from there, so that a wave waits for two reads of the
// arguments.  (A search by halves waits for eight: 400 tensors of 61M elements 202
// us instead of 200, read back 129 instead of 127; the lanes of a wave looking at
// all at once wait for vector loads: 204 and 157.)
template <class A>
__device__ __forceinline__ int piece_of(A a, uint32_t tile) {
    if (a->n == 1) return 0;
    int t = 0;
#pragma unroll
    for (int k = 16; k < a->kRows; k += 16) t += a->first_tile[k] <= tile ? 16 : 0;
    const auto* const some = &a->first_tile[t];
#pragma unroll
    for (int k = 1; k < 16; ++k) t += some[k] <= tile ? 1 : 0;
    return t;
}

// One tensor's streams.
struct Streams {
    const char* g;
    char* w;
    char* m;
    char* v;
    char* s;
    char* p;
    int64_t n;
};
// What a lane holds of a span.
struct Lane {
    u32x4 g, w;
    uint32_t m, v, s;
};

template <bool GB, bool WHOLE>
__device__ __forceinline__ Lane load_lane(const Streams& x, int64_t at) {
    const int64_t i = at + mx::lane_id() * 4;
    Lane l;
    if constexpr (WHOLE) {
        if constexpr (GB) {
            const u32x2 h = gv::load2_nt(x.g + i * 2);
            l.g = u32x4{h[0], h[1], 0u, 0u};
        } else {
            l.g = gv::load4_nt(x.g + i * 4);
        }
        l.w = gv::load4_nt(x.w + i * 4);
    } else {
        l.g = gv::load_some<GB, 4>(x.g, i, x.n);
        l.w = gv::load_some<false, 4>(x.w, i, x.n);
    }
    l.m = load_bytes<WHOLE>(x.m, i, x.n);
    l.v = load_bytes<WHOLE>(x.v, i, x.n);
    const int64_t b = i / kBlockElems;
    l.s = WHOLE || b * kBlockElems < x.n ? *reinterpret_cast<const uint16_t*>(x.s + b * 2) : 0u;
    return l;
}

template <bool GB, int PM, bool WHOLE>
__device__ __forceinline__ void step_lane(const Streams& x, int64_t at, const Lane& l, const adamw::Factors& f,
                                          uint32_t key) {
    const int64_t i = at + mx::lane_id() * 4;
    const float ms = mx::scale_of(l.s & 0xffu);
    const float vs = mx::scale_of(l.s >> 8);
    const mx::f32x2 m01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(l.m, ms, false);
    const mx::f32x2 m23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(l.m, ms, true);
    float me[4] = {m01[0], m01[1], m23[0], m23[1]};
    float ve[4], wn[4];
    uint32_t mtop = 0, vtop = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        ve[e] = decode_v((l.v >> (8 * e)) & 0xffu, vs);
        adamw::adamw_moments(rr::elem<GB>(l.g, e), me[e], ve[e], f);
        wn[e] = step_weight(__uint_as_float(l.w[e]), me[e], ve[e], f);
        if (WHOLE || i + e < x.n) {
            mtop = mx::larger(mtop, __float_as_uint(me[e]) & 0x7fffffffu);
            vtop = mx::larger(vtop, __float_as_uint(ve[e]));     // no sign, but for a NaN's
        }
    }
    const uint32_t sm = scale_m(mx::max_of_8(mtop));
    const uint32_t sv = scale_v(mx::max_of_8(vtop));
    const float up = __uint_as_float((254u - (sm < 254u ? sm : 254u)) << 23);
    const uint32_t from = 8u - ((sv - 31u) << 23);
    const uint32_t x0 = key + static_cast<uint32_t>(i) * kGolden;
    uint32_t mt[4], vt[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t r = random_bits(x0 + e * kGolden);
        mt[e] = encode_m(me[e], up, r);
        vt[e] = encode_v(ve[e], from, r);
    }
    const uint32_t mc = sm == 255u ? 0x7f7f7f7fu : top_bytes(mt);
    const uint32_t vc = sv == 255u || sv == 0u ? 0u : top_bytes(vt);
    store_bytes<WHOLE>(x.m, i, x.n, mc);
    store_bytes<WHOLE>(x.v, i, x.n, vc);
    const int64_t b = i / kBlockElems;
    if ((threadIdx.x & 7) == 0 && (WHOLE || b * kBlockElems < x.n))
        *reinterpret_cast<uint16_t*>(x.s + b * 2) = static_cast<uint16_t>(sm | sv << 8);
    const u32x4 wq = {__float_as_uint(wn[0]), __float_as_uint(wn[1]), __float_as_uint(wn[2]), __float_as_uint(wn[3])};
    const u32x2 h = {mx::pack_bf16(wn[0], wn[1]), mx::pack_bf16(wn[2], wn[3])};
    if constexpr (WHOLE) {
        gv::store4_nt(x.w + i * 4, wq);
        if constexpr (PM == 1) gv::store4_nt(x.p + i * 4, wq);
        if constexpr (PM == 2) gv::store2_nt(x.p + i * 2, h);
    } else {
        gv::store_some<false, 4>(x.w, i, x.n, wq);
        if constexpr (PM == 1) gv::store_some<false, 4>(x.p, i, x.n, wq);
        if constexpr (PM == 2) gv::store_some<true, 4>(x.p, i, x.n, u32x4{h[0], h[1], 0u, 0u});
    }
}

// GB: bf16 gradients.  PM: the copy, 0 none, 1 float32, 2 bf16.
template <bool GB, int PM, int U>
__global__ __launch_bounds__(kLanes) void adamw8_kernel(Adam8Args<PM != 0>) {
    typedef const __attribute__((address_space(4))) Adam8Args<PM != 0>* KAdam8;
    const KAdam8 a = (KAdam8)(__builtin_amdgcn_kernarg_segment_ptr());
    const uint32_t tiles = a->tiles;
    const adamw::KScalars k = (adamw::KScalars)(&a->scalars);
    const float norm = k->norm != nullptr ? gv::load_uniform(k->norm) : 0.0f;
    const int64_t step = k->step != nullptr ? gv::load_uniform(k->step) : k->host_step;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int t = piece_of(a, tile);
        const Streams x = {a->g[t], a->w[t], a->m[t], a->v[t], a->s[t], PM != 0 ? a->p[PM != 0 ? t : 0] : nullptr,
                           a->count[t]};
        const int64_t at = (static_cast<int64_t>(tile - a->first_tile[t]) * 4 + wave) * (U * kSpan);
        const bool whole = at + U * kSpan <= x.n;
        Lane l[U];
        if (whole) {
#pragma unroll
            for (int u = 0; u < U; ++u) l[u] = load_lane<GB, true>(x, at + u * kSpan);
        }
        // The factors (divisions, two powers) and the key while the data is in
        // flight.
        adamw::Factors f;
        if (!adamw::factors(k, norm, step, f)) return;
        uint32_t key = mix_word(a->seed, static_cast<uint32_t>(step));
        key = mix_word(key, static_cast<uint32_t>(step >> 32));
        key = mix_word(mix_word(key, a->tensor + t), a->piece);
        if (whole) {
#pragma unroll
            for (int u = 0; u < U; ++u) step_lane<GB, PM, true>(x, at + u * kSpan, l[u], f, key);
        } else {
            for (int64_t i = at; i < x.n && i < at + U * kSpan; i += kSpan)
                step_lane<GB, PM, false>(x, i, load_lane<GB, false>(x, i), f, key);
        }
    }
}

template <int U>
const void* kernel_for(const AdamWLaunch& l) {
    const int pm = l.params == nullptr ? 0 : (l.param_bf16 ? 2 : 1);
    if (l.grad_bf16) {
        return pm == 0 ? reinterpret_cast<const void*>(&adamw8_kernel<true, 0, U>)
               : pm == 1 ? reinterpret_cast<const void*>(&adamw8_kernel<true, 1, U>)
                         : reinterpret_cast<const void*>(&adamw8_kernel<true, 2, U>);
    }
    return pm == 0 ? reinterpret_cast<const void*>(&adamw8_kernel<false, 0, U>)
           : pm == 1 ? reinterpret_cast<const void*>(&adamw8_kernel<false, 1, U>)
                     : reinterpret_cast<const void*>(&adamw8_kernel<false, 2, U>);
}

// The moments' values.
constexpr int read_spans(bool bf16) { return bf16 ? 2 : 1; }
struct Read8Args {
    static constexpr int kCap = 163, kRows = rows_for(kCap);
    const char* m[kCap];
    const char* v[kCap];
    const char* s[kCap];
    char* m_out[kCap];
    char* v_out[kCap];
    uint32_t count[kCap];
    uint32_t first_tile[kRows];    // behind the last tensor none that a tile can have
    int32_t n;
    uint32_t tiles;
};
static_assert(sizeof(Read8Args) <= kArgBytes, "kernel arguments");
typedef const __attribute__((address_space(4))) Read8Args* KRead8;

// A lane's 8 elements of a span of 512 (mx.h: wide for float32 outputs).
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void load_moments(const char* m, const char* v, const char* s, int64_t at, int64_t n,
                                             u32x2& mq, u32x2& vq, uint32_t& sq) {
    const int64_t i = mx::first4<!BF16>(at), j = i + mx::second_after(!BF16);
    mq = u32x2{load_bytes<WHOLE>(m, i, n), load_bytes<WHOLE>(m, j, n)};
    vq = u32x2{load_bytes<WHOLE>(v, i, n), load_bytes<WHOLE>(v, j, n)};
    const int64_t b = at / kBlockElems + mx::scale_place<!BF16>();
    sq = WHOLE || b * kBlockElems < n ? *reinterpret_cast<const uint16_t*>(s + b * 2) : 0u;
}
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store_moments(char* m_out, char* v_out, int64_t at, int64_t n, u32x2 mq, u32x2 vq,
                                              uint32_t sq) {
    float m[8], v[8];
    const mx::Scales s = mx::own_scales<!BF16>(sq);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float ms = mx::scale_of((h == 0 ? s.a : s.b) & 0xffu);
        const float vs = mx::scale_of((h == 0 ? s.a : s.b) >> 8);
        const mx::f32x2 m01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(mq[h], ms, false);
        const mx::f32x2 m23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(mq[h], ms, true);
        m[4 * h] = m01[0], m[4 * h + 1] = m01[1], m[4 * h + 2] = m23[0], m[4 * h + 3] = m23[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * h + e] = decode_v((vq[h] >> (8 * e)) & 0xffu, vs);
    }
    mx::store_values<BF16, !BF16, WHOLE>(m_out, at, n, m);
    mx::store_values<BF16, !BF16, WHOLE>(v_out, at, n, v);
}

template <bool BF16>
__global__ __launch_bounds__(kLanes) void adamw8_read_kernel(Read8Args) {
    constexpr int U = read_spans(BF16);
    const KRead8 a = (KRead8)(__builtin_amdgcn_kernarg_segment_ptr());
    const uint32_t tiles = a->tiles;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int t = piece_of(a, tile);
        const char* const m = a->m[t];
        const char* const v = a->v[t];
        const char* const s = a->s[t];
        const int64_t n = a->count[t];
        const int64_t at = mx::wave_start<U>(tile - a->first_tile[t]);
        u32x2 mq[U], vq[U];
        uint32_t sq[U];
        if (at + U * mx::kMxSpan <= n) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                load_moments<BF16, true>(m, v, s, at + u * mx::kMxSpan, n, mq[u], vq[u], sq[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                store_moments<BF16, true>(a->m_out[t], a->v_out[t], at + u * mx::kMxSpan, n, mq[u], vq[u], sq[u]);
        } else {
            for (int64_t i = at; i < n && i < at + U * mx::kMxSpan; i += mx::kMxSpan) {
                load_moments<BF16, false>(m, v, s, i, n, mq[0], vq[0], sq[0]);
                store_moments<BF16, false>(a->m_out[t], a->v_out[t], i, n, mq[0], vq[0], sq[0]);
            }
        }
    }
}

int launch(const void* fn, void* args, uint32_t tiles, unsigned lds, void* stream, const char* what, const char** msg) {
    void* list[] = {args};
    const hipError_t e = hipLaunchKernel(fn, dim3(std::min(tiles, kMaxGrid)), dim3(kLanes), list, lds,
                                         static_cast<hipStream_t>(stream));
    if (e == hipSuccess) return 0;
    *msg = what;
    return static_cast<int>(e);
}

// A launch's tensors, from tensor t on: fill(slot, tensor, first element)
// for each, until the arguments are full or a tensor is too long for one launch,
// whose pieces (`at`: the next one's first element) go alone.
template <class A, class F>
void fill_launch(A& a, int32_t n_tensors, const int64_t* numels, int64_t tile, int32_t& t, int64_t& at, F fill) {
    int64_t tiles = 0;
    for (a.n = 0; t < n_tensors && a.n < A::kCap;) {
        const bool alone = numels[t] > kMaxPiece;
        if (alone && a.n > 0) break;
        const int64_t count = std::min(numels[t] - at, kMaxPiece);
        fill(a.n, t, at);
        a.count[a.n] = static_cast<uint32_t>(count);
        a.first_tile[a.n] = static_cast<uint32_t>(tiles);
        tiles += (count + tile - 1) / tile;
        ++a.n;
        at += count;
        if (at >= numels[t]) {
            ++t;
            at = 0;
        }
        if (alone) break;
    }
    a.tiles = static_cast<uint32_t>(tiles);
    std::fill(a.first_tile + a.n, a.first_tile + A::kRows, UINT32_MAX);
}

template <bool PARAMS>
int launch_step(const AdamW8Launch& l, const char** msg) {
    const AdamWLaunch& b = l.step;
    Adam8Args<PARAMS> a;
    a.scalars = adamw::scalars_of(b);
    a.seed = mix_word(mix_word(0, static_cast<uint32_t>(l.seed)), static_cast<uint32_t>(l.seed >> 32));
    int64_t all = 0;
    for (int32_t t = 0; t < b.n_tensors && all <= kMxShort; ++t) all += b.numels[t];
    const int spans = all <= kMxShort ? 1 : kSpans;
    const void* fn = spans == 1 ? kernel_for<1>(b) : kernel_for<kSpans>(b);
    int64_t at = 0;
    for (int32_t t = 0; t < b.n_tensors;) {
        a.tensor = static_cast<uint32_t>(t);
        a.piece = static_cast<uint32_t>(at / kMaxPiece);
        fill_launch(a, b.n_tensors, b.numels, 4 * spans * kSpan, t, at, [&](int k, int32_t i, int64_t from) {
            a.g[k] = static_cast<const char*>(b.grads[i]) + from * (b.grad_bf16 ? 2 : 4);
            a.w[k] = reinterpret_cast<char*>(b.w[i] + from);
            a.m[k] = reinterpret_cast<char*>(l.m[i] + from);
            a.v[k] = reinterpret_cast<char*>(l.v[i] + from);
            a.s[k] = reinterpret_cast<char*>(l.scales[i] + from / kBlockElems * 2);
            if constexpr (PARAMS) a.p[k] = static_cast<char*>(b.params[i]) + from * (b.param_bf16 ? 2 : 4);
        });
        if (a.tiles == 0) continue;
        if (const int e = launch(fn, &a, a.tiles, lds_reserve(kAdamW8WgPerCu), b.stream, "hipLaunchKernel(adamw8)", msg))
            return e;
    }
    return 0;
}

}  // namespace

int launch_adamw8(const AdamW8Launch& l, const char** msg) {
    return l.step.params != nullptr ? launch_step<true>(l, msg) : launch_step<false>(l, msg);
}

int launch_adamw8_read(const Moments8Read& l, const char** msg) {
    Read8Args a;
    const void* fn = l.out_bf16 ? reinterpret_cast<const void*>(&adamw8_read_kernel<true>)
                                : reinterpret_cast<const void*>(&adamw8_read_kernel<false>);
    const int64_t es = l.out_bf16 ? 2 : 4;
    int64_t at = 0;
    for (int32_t t = 0; t < l.n_tensors;) {
        fill_launch(a, l.n_tensors, l.numels, 2048 * read_spans(l.out_bf16), t, at,
                    [&](int k, int32_t i, int64_t from) {
                        a.m[k] = reinterpret_cast<const char*>(l.m[i] + from);
                        a.v[k] = reinterpret_cast<const char*>(l.v[i] + from);
                        a.s[k] = reinterpret_cast<const char*>(l.scales[i] + from / kBlockElems * 2);
                        a.m_out[k] = static_cast<char*>(l.m_out[i]) + from * es;
                        a.v_out[k] = static_cast<char*>(l.v_out[i]) + from * es;
                    });
        if (a.tiles == 0) continue;
        if (const int e = launch(fn, &a, a.tiles, lds_reserve(kMoments8WgPerCu), l.stream, "hipLaunchKernel(adamw8_read)",
                                 msg))
            return e;
    }
    return 0;
}

}  // namespace ddp

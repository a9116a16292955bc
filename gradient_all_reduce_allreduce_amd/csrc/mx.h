// mx.h -- device helpers of the kernels on microscaled gradients and 8-bit
// moments (mx4.hip, mx4_reduce.hip, adamw8.hip).
//
// A block is 32 consecutive elements with one scale byte s, which stands for
// 2^(s - 127) (255: the block holds no numbers).  An element of 4 bits is
// sign, 2 bits of exponent, 1 of mantissa: 0, .5, 1, 1.5, 2, 3, 4, 6; element
// 2k of a row is the low half of byte k.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grad_vec.h"

namespace ddp {
namespace mx {

using rr::u32x2;
using rr::u32x4;

constexpr int kMxBlock = 32;
constexpr int kWave = 64;

typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int CTRL>
__device__ __forceinline__ uint32_t lane(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest over a quad of lanes, and over 8 lanes, in each of them: the
// neighbour, the other pair, the other quad (which a mirror of 8 lanes reaches,
// its lanes being equal by then).
__device__ __forceinline__ uint32_t max_of_4(uint32_t x) {
    x = larger(x, lane<0xB1>(x));
    return larger(x, lane<0x4E>(x));
}
__device__ __forceinline__ uint32_t max_of_8(uint32_t x) {
    x = max_of_4(x);
    return larger(x, lane<0x141>(x));
}

// A scale byte as the conversions take it, the power of two as a float32: they
// read the exponent's bits only (0: 2^-127; all ones: every result is NaN).
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s << 23); }

// 8 codes as 8 values.
__device__ __forceinline__ void decode8(uint32_t codes, float scale, float (&x)[8]) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
    x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
}
// 8 values, in scales, to the nearest codes (ties to even).
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float scale) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], scale, 3);
}

// Quantisation of a block held by a quad of lanes, 8 elements each.  The scale
// is the smallest power of two that lets no element round past the top level
// 6: with the block's maximum rounded to one bit of mantissa (nearest, a tie up)
// its exponent less 2, and 2^-126 at least, so that it is a normal float32.
// Every element is then off by half a step at most, the largest ones too.
// A maximum of 1.75 * 2^127 or more (its level would not be a float32), an
// infinity or a NaN makes the whole block NaN.
struct Coded {
    uint32_t codes;
    uint32_t scale;     // the byte
    bool finite;
};
__device__ __forceinline__ Coded quantize8(const float (&x)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = larger(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = max_of_4(top) + 0x200000u;
    Coded q;
    q.finite = top < 0x7f800000u;
    const uint32_t e = top >> 23;
    q.scale = larger(e, 3u) - 2u;
    q.codes = encode8(x, scale_of(q.scale));
    if (!q.finite) {
        q.codes = 0;
        q.scale = 255;
    }
    return q;
}

// A lane's 8 consecutive elements as values, and back.
template <bool BF16>
struct Oct {
    u32x4 lo, hi;      // bf16: hi unused
};
template <bool BF16>
__device__ __forceinline__ float oct_elem(const Oct<BF16>& o, int e) {
    if constexpr (BF16) return rr::elem<true>(o.lo, e);
    return __uint_as_float(e < 4 ? o.lo[e & 3] : o.hi[e & 3]);
}
template <bool BF16>
__device__ __forceinline__ Oct<BF16> pack_oct(const float (&x)[8]) {
    Oct<BF16> o;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (BF16) {
            o.lo[k] = rr::bf16_bits(x[2 * k]) | (rr::bf16_bits(x[2 * k + 1]) << 16);
        } else {
            o.lo[k] = __float_as_uint(x[k]);
            o.hi[k] = __float_as_uint(x[4 + k]);
        }
    }
    return o;
}
// The elements i .. i + 7 of a row (`whole`: all of them lie in it), zero
// where there are none.
template <bool BF16>
__device__ __forceinline__ Oct<BF16> load_oct(const char* p, int64_t i, int64_t n, bool whole) {
    Oct<BF16> o;
    if (whole) {
        if constexpr (BF16) {
            o.lo = gv::load4_nt(p + i * 2);
        } else {
            o.lo = gv::load4_nt(p + i * 4);
            o.hi = gv::load4_nt(p + i * 4 + 16);
        }
    } else if constexpr (BF16) {
        o.lo = gv::load_some<true, 8>(p, i, n);
    } else {
        o.lo = gv::load_some<false, 4>(p, i, n);
        o.hi = gv::load_some<false, 4>(p, i + 4, n);
    }
    return o;
}
template <bool BF16>
__device__ __forceinline__ void store_oct(char* p, int64_t i, int64_t n, bool whole, const Oct<BF16>& o) {
    if (whole) {
        if constexpr (BF16) {
            gv::store4_nt(p + i * 2, o.lo);
        } else {
            gv::store4_nt(p + i * 4, o.lo);
            gv::store4_nt(p + i * 4 + 16, o.hi);
        }
    } else if constexpr (BF16) {
        gv::store_some<true, 8>(p, i, n, o.lo);
    } else {
        gv::store_some<false, 4>(p, i, n, o.lo);
        gv::store_some<false, 4>(p, i + 4, n, o.hi);
    }
}

// Codes (4 bytes per lane) and scale bytes of a row.
typedef __attribute__((address_space(1))) const uint32_t* GlobalCodes;
typedef __attribute__((address_space(1))) uint32_t* GlobalCodesOut;
typedef __attribute__((address_space(1))) const uint8_t* GlobalBytes;
typedef __attribute__((address_space(1))) uint8_t* GlobalBytesOut;

__device__ __forceinline__ uint32_t load_codes(const char* p, int64_t i) {
    return __builtin_nontemporal_load((GlobalCodes)(p + i / 2));
}
__device__ __forceinline__ void store_codes(char* p, int64_t i, uint32_t c) {
    __builtin_nontemporal_store(c, (GlobalCodesOut)(p + i / 2));
}
__device__ __forceinline__ uint32_t load_scale(const char* p, int64_t i) { return *(GlobalBytes)(p + i / kMxBlock); }
__device__ __forceinline__ void store_scale(char* p, int64_t i, uint32_t s) {
    *(GlobalBytesOut)(p + i / kMxBlock) = static_cast<uint8_t>(s);
}

}  // namespace mx
}  // namespace ddp

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
constexpr int kMxSpan = 512;      // elements a wave takes at once

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

// Two float32 as bf16, nearest even, the first in the low half; a NaN stays
// one.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// A scale byte as the conversions take it, the power of two as a float32: they
// read the exponent's bits only (0: 2^-127; all ones: every result is NaN).
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s << 23); }

// How the kernels walk over a row: workgroups of 4 waves, every wave takes U
// spans of 512 consecutive elements, a lane 8 elements of each.  What is 2 or
// less bytes an element goes naturally, the 8 elements consecutive: 4 bytes of
// codes, 16 of bf16, a quad of lanes a block.  Of float32 a lane would reach
// over 32 bytes, and an instruction would write every line by halves (which
// reach memory as halves when the second one comes late: decoding 8 rows to
// float32 took 1.6 times as long).  So float32 goes WIDE: lane l holds the
// elements 4l .. 4l + 3 and 256 + 4l .. 256 + 4l + 3 of the span, 16 bytes of
// consecutive kilobytes, 8 lanes a block.  Quantisation and the moments' reading
// are wide as wholes where float32 is among their rows, and a pair of lanes shares
// two dwords of codes, or two blocks' scales, which it exchanges in registers;
// kernels that load codes load them naturally and exchange the values through LDS.
constexpr int kMxWaves = 4;

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// Where the lane's first and second four elements lie in the span at `at`.
template <bool WIDE>
__device__ __forceinline__ int64_t first4(int64_t at) {
    return at + lane_id() * (WIDE ? 4 : 8);
}
constexpr int second_after(bool wide) { return wide ? 256 : 4; }

// Where this lane's dword of codes and its scale byte lie in the span; WIDE (codes
// are only stored so): even lanes have those of the first four elements of both
// lanes of a pair, odd lanes those of the second.
template <bool WIDE>
__device__ __forceinline__ int code_place() {      // in bytes
    const int l = lane_id();
    return 4 * (WIDE ? (l >> 1) + (l & 1) * 32 : l);
}
template <bool WIDE>
__device__ __forceinline__ int scale_place() {
    const int l = lane_id();
    return WIDE ? (l >> 3) + (l & 1) * 8 : l >> 2;
}

// From the codes of this lane's own 8 elements to that dword.
__device__ __forceinline__ uint32_t halves() { return (lane_id() & 1) ? 0x07060302u : 0x05040100u; }
template <bool WIDE>
__device__ __forceinline__ uint32_t shared_codes(uint32_t c) {
    return WIDE ? __builtin_amdgcn_perm(lane<0xF5>(c), lane<0xA0>(c), halves()) : c;
}

// The scales of a lane's first and second four elements.
struct Scales {
    uint32_t a, b;      // the bytes
};
template <bool WIDE>
__device__ __forceinline__ Scales own_scales(uint32_t s) {
    if constexpr (WIDE) return {lane<0xA0>(s), lane<0xF5>(s)};
    return {s, s};
}

// 8 codes as 8 values.
__device__ __forceinline__ void decode8(uint32_t codes, Scales s, float (&x)[8]) {
    const float sa = scale_of(s.a), sb = scale_of(s.b);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sa, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sa, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sb, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sb, 3);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
    x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
}
// 8 values, in scales, to the nearest codes (ties to even).
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], Scales s) {
    const float sa = scale_of(s.a), sb = scale_of(s.b);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], sa, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], sa, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], sb, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], sb, 3);
}

// Quantisation of the blocks that a quad of lanes (WIDE: two that 8 lanes)
// holds.  The scale is the smallest power of two that lets no element round past
// the top level 6: with the block's maximum rounded to one bit of mantissa
// (nearest, a tie up) its exponent less 2, and 2^-126 at least, so that it is a
// normal float32.  Every element is then off by half a step at most, the largest
// ones too.  A maximum of 1.75 * 2^127 or more (its level would not be a
// float32), an infinity or a NaN makes the whole block NaN.
struct Coded {
    uint32_t codes;     // of the lane's own elements
    Scales scales;
    bool finite_a, finite_b;
};
template <bool WIDE>
__device__ __forceinline__ Coded quantize8(const float (&x)[8]) {
    uint32_t ta = 0, tb = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        ta = larger(ta, __float_as_uint(x[e]) & 0x7fffffffu);
        tb = larger(tb, __float_as_uint(x[4 + e]) & 0x7fffffffu);
    }
    if constexpr (WIDE) {
        ta = max_of_8(ta), tb = max_of_8(tb);
    } else {
        ta = tb = max_of_4(larger(ta, tb));
    }
    ta += 0x200000u, tb += 0x200000u;
    Coded q;
    q.finite_a = ta < 0x7f800000u;
    q.finite_b = tb < 0x7f800000u;
    q.scales = {larger(ta >> 23, 3u) - 2u, larger(tb >> 23, 3u) - 2u};
    q.codes = encode8(x, q.scales);
    if (!q.finite_a) {
        q.codes &= WIDE ? 0xffff0000u : 0u;
        q.scales.a = 255;
    }
    if (!q.finite_b) {
        q.codes &= WIDE ? 0x0000ffffu : 0u;
        q.scales.b = 255;
    }
    return q;
}

// A lane's 8 values as they lie in memory: natural bf16 8 consecutive ones in
// a; WIDE four in each (bf16: in the lower halves of a and b).
struct Raw {
    u32x4 a, b;
};
template <bool BF16, bool WIDE, bool WHOLE>
__device__ __forceinline__ Raw load_raw(const char* p, int64_t at, int64_t n) {
    static_assert(BF16 || WIDE, "float32 is wide");
    const int64_t i = first4<WIDE>(at);
    Raw x{};
    if constexpr (!WIDE) {
        x.a = WHOLE ? gv::load4_nt(p + i * 2) : gv::load_some<true, 8>(p, i, n);
    } else if constexpr (!WHOLE) {
        x.a = gv::load_some<BF16, 4>(p, i, n);
        x.b = gv::load_some<BF16, 4>(p, i + 256, n);
    } else if constexpr (BF16) {
        const u32x2 a = gv::load2_nt(p + i * 2), b = gv::load2_nt(p + i * 2 + 512);
        x.a = u32x4{a[0], a[1], 0u, 0u};
        x.b = u32x4{b[0], b[1], 0u, 0u};
    } else {
        x.a = gv::load4_nt(p + i * 4);
        x.b = gv::load4_nt(p + i * 4 + 1024);
    }
    return x;
}
// The elements i .. i + 3 of a row in registers' order.
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store4(char* p, int64_t i, int64_t n, const float* x) {
    u32x4 v = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    if constexpr (BF16) {
        v = u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), 0u, 0u};
    }
    if constexpr (!WHOLE) {
        gv::store_some<BF16, 4>(p, i, n, v);
    } else if constexpr (BF16) {
        gv::store2_nt(p + i * 2, u32x2{v[0], v[1]});
    } else {
        gv::store4_nt(p + i * 4, v);
    }
}
template <bool BF16, bool WIDE, bool WHOLE>
__device__ __forceinline__ void store_values(char* p, int64_t at, int64_t n, const float (&x)[8], bool keep_a = true,
                                             bool keep_b = true) {
    static_assert(BF16 || WIDE, "float32 is wide");
    const int64_t i = first4<WIDE>(at);
    if constexpr (!WIDE) {
        u32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
        if (!keep_a) return;
        if constexpr (WHOLE) gv::store4_nt(p + i * 2, v);
        else gv::store_some<true, 8>(p, i, n, v);
    } else {
        if (keep_a) store4<BF16, WHOLE>(p, i, n, &x[0]);
        if (keep_b) store4<BF16, WHOLE>(p, i + 256, n, &x[4]);
    }
}
template <bool BF16, bool WIDE>
__device__ __forceinline__ void values_of(const Raw& r, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = WIDE ? rr::elem<BF16>(e < 4 ? r.a : r.b, e & 3) : rr::elem<BF16>(r.a, e);
}
// A lane's 8 consecutive values to the wide places and back, through 2 KiB of
// LDS of the wave's own.  (Its lanes run together and its LDS operations in
// order; the fences keep the compiler from changing that order.)
struct Exchange {
    u32x4 slot[kMxWaves][128];
};
constexpr unsigned kExchangeBytes = sizeof(Exchange);
// A kernel's area; null for kernels that do not exchange.
template <bool NEEDED>
__device__ __forceinline__ Exchange* exchange_area() {
    if constexpr (NEEDED) {
        __shared__ Exchange area;
        return &area;
    } else {
        return nullptr;
    }
}
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
template <bool TO_WIDE>
__device__ __forceinline__ void exchange(Exchange& lds, float (&x)[8]) {
    u32x4* const s = lds.slot[threadIdx.x >> 6];
    const int l = lane_id();
    const u32x4 a = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    const u32x4 b = {__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])};
    wave_order();
    s[TO_WIDE ? 2 * l : l] = a;
    s[TO_WIDE ? 2 * l + 1 : 64 + l] = b;
    wave_order();
    const u32x4 c = s[TO_WIDE ? l : 2 * l];
    const u32x4 d = s[TO_WIDE ? 64 + l : 2 * l + 1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = __uint_as_float(c[e]);
        x[4 + e] = __uint_as_float(d[e]);
    }
}

// Whether element e of the lane lies in the row.
template <bool WIDE>
__device__ __forceinline__ bool in_row(int64_t at, int64_t n, int e) {
    return first4<WIDE>(at) + (e & 3) + (e < 4 ? 0 : second_after(WIDE)) < n;
}

// A lane's dword of codes and its scale byte.  Codes end with the row's last
// block.
typedef __attribute__((address_space(1))) const uint32_t* GlobalCodes;
typedef __attribute__((address_space(1))) uint32_t* GlobalCodesOut;
typedef __attribute__((address_space(1))) const uint8_t* GlobalBytes;
typedef __attribute__((address_space(1))) uint8_t* GlobalBytesOut;

// Whether that dword's block has elements of the row.
template <bool WIDE, bool WHOLE>
__device__ __forceinline__ bool block_in_row(int64_t at, int64_t n) {
    return WHOLE || at + scale_place<WIDE>() * kMxBlock < n;
}
// (Loaded naturally by every kernel.)
template <bool WHOLE>
__device__ __forceinline__ uint32_t load_codes(const char* p, int64_t at, int64_t n) {
    return block_in_row<false, WHOLE>(at, n) ? __builtin_nontemporal_load((GlobalCodes)(p + at / 2 + code_place<false>())) : 0u;
}
template <bool WHOLE>
__device__ __forceinline__ uint32_t load_scale(const char* p, int64_t at, int64_t n) {
    return block_in_row<false, WHOLE>(at, n) ? *(GlobalBytes)(p + at / kMxBlock + scale_place<false>()) : 0u;
}
// `c`: shared_codes of the lane's own.
template <bool WIDE, bool WHOLE>
__device__ __forceinline__ void store_coded(char* codes, char* scales, int64_t at, int64_t n, uint32_t c, Scales s) {
    if (!block_in_row<WIDE, WHOLE>(at, n)) return;
    __builtin_nontemporal_store(c, (GlobalCodesOut)(codes + at / 2 + code_place<WIDE>()));
    // the first lane of a block, or pair of lanes of two
    if ((threadIdx.x & (WIDE ? 6 : 3)) == 0)
        *(GlobalBytesOut)(scales + at / kMxBlock + scale_place<WIDE>()) =
            static_cast<uint8_t>(WIDE && (threadIdx.x & 1) ? s.b : s.a);
}

// This wave's first element in workgroup-sized piece `tile` of a row.
template <int U>
__device__ __forceinline__ int64_t wave_start(uint32_t tile) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return (static_cast<int64_t>(tile) * kMxWaves + wave) * (kMxSpan * U);
}

}  // namespace mx
}  // namespace ddp

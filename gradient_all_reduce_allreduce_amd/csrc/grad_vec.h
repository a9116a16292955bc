// grad_vec.h -- device helpers shared by the kernels that walk many gradient
// tensors (grad_norm.hip, adamw.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ring_reduce_impl.h"

namespace ddp {
namespace gv {

using rr::u32x2;
using rr::u32x4;

// Vectors at addresses aligned to the element only.  The hardware's vector
// accesses take any alignment, so a tensor whose start differs from the
// others' within 16 bytes needs no path of its own; aligned ones compile
// to the same instruction.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;
// Through global-address-space pointers: the tensors' addresses come out of
// an argument table, where the compiler cannot tell that they are global.
typedef __attribute__((address_space(1))) const u32x4_any* GlobalIn4;
typedef __attribute__((address_space(1))) const u32x2_any* GlobalIn2;
typedef __attribute__((address_space(1))) u32x4_any* GlobalOut4;
typedef __attribute__((address_space(1))) u32x2_any* GlobalOut2;

__device__ __forceinline__ u32x4 load4(const char* p) { return *(GlobalIn4)(p); }
__device__ __forceinline__ u32x2 load2(const char* p) { return *(GlobalIn2)(p); }
__device__ __forceinline__ u32x4 load4_nt(const char* p) { return __builtin_nontemporal_load((GlobalIn4)(p)); }
__device__ __forceinline__ u32x2 load2_nt(const char* p) { return __builtin_nontemporal_load((GlobalIn2)(p)); }
__device__ __forceinline__ void store4_nt(char* p, u32x4 v) { __builtin_nontemporal_store(v, (GlobalOut4)(p)); }
__device__ __forceinline__ void store2_nt(char* p, u32x2 v) { __builtin_nontemporal_store(v, (GlobalOut2)(p)); }

// The elements k .. k + N - 1 of a vector's lane that lie in [0, n), element 0
// at p: the loads of a tensor's first and last vector, all in flight at once,
// zero in the other places; and the stores.
template <bool BF16, int N>
__device__ __forceinline__ u32x4 load_some(const char* p, int64_t k, int64_t n) {
    u32x4 x = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < N; ++e) {
        uint32_t b = 0;
        if (k + e >= 0 && k + e < n) {
            if constexpr (BF16) {
                b = *reinterpret_cast<const uint16_t*>(p + (k + e) * 2);
            } else {
                b = *reinterpret_cast<const uint32_t*>(p + (k + e) * 4);
            }
        }
        if constexpr (BF16) {
            x[e / 2] |= b << (16 * (e & 1));
        } else {
            x[e] = b;
        }
    }
    return x;
}
template <bool BF16, int N>
__device__ __forceinline__ void store_some(char* p, int64_t k, int64_t n, const u32x4& x) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (k + e < 0 || k + e >= n) continue;
        if constexpr (BF16) {
            *reinterpret_cast<uint16_t*>(p + (k + e) * 2) = static_cast<uint16_t>(x[e / 2] >> (16 * (e & 1)));
        } else {
            *reinterpret_cast<uint32_t*>(p + (k + e) * 4) = x[e];
        }
    }
}

// A value that every lane reads and that no kernel running now writes, through
// the constant address space: a scalar load.  Through a plain pointer the
// compiler cannot rule out the kernel's own stores and takes a vector load,
// which would wait behind the tile's data.
template <class T>
__device__ __forceinline__ T load_uniform(const T* p) {
    return *(const __attribute__((address_space(4))) T*)(p);
}

// The clipping factor min(1, max_norm / (norm + 1e-6)) in float32, one
// rounding per operation.  No limit (infinite max_norm) never scales; a
// norm that is infinite gives 0 and one that is NaN gives NaN.
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
#pragma clang fp contract(off)
    if (max_norm == __builtin_inff()) return 1.0f;
    const float c = max_norm / (norm + 1e-6f);
    return c > 1.0f ? 1.0f : c;
}

// x plus the value of another lane, chosen by a data-parallel-primitive
// control; lanes it does not reach add zero.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_lane(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xf, true);
    return x + __builtin_bit_cast(double, lo | static_cast<uint64_t>(hi) << 32);
}

// The sum over the wave's lanes in a fixed order, in lane 63: shifts by 1, 2,
// 4 and 8 within each row of 16 lanes, then row sums into the next row and
// the lower half's into the upper.  In registers, where exchanging lanes
// through the LDS crossbar would wait a round trip for each of six steps.
__device__ __forceinline__ double wave_sum63(double x) {
    x = add_lane<0x111, 0xf>(x);
    x = add_lane<0x112, 0xf>(x);
    x = add_lane<0x114, 0xf>(x);
    x = add_lane<0x118, 0xf>(x);
    x = add_lane<0x142, 0xa>(x);
    return add_lane<0x143, 0xc>(x);
}

// The sum over the workgroup in a fixed order, in every lane.  Once per
// kernel: a second call would need a barrier before it.
template <int BLOCK>
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[BLOCK / 64];
    x = wave_sum63(x);
    if ((threadIdx.x & 63) == 63) part[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = part[0];
#pragma unroll
    for (int w = 1; w < BLOCK / 64; ++w) s += part[w];
    return s;
}

}  // namespace gv
}  // namespace ddp

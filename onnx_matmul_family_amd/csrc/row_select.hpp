// Ordering of floats by value for selections ("the k largest, ties to the
// lowest index") and wave-wide reductions, shared by the router and the token
// log-probability kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace omm {

// kind: 0 = bf16, 1 = fp16, 2 = fp32
template <int DT> struct elem_of { typedef uint16_t type; };
template <> struct elem_of<2> { typedef float type; };

template <int DT>
__device__ __forceinline__ float elem_f32(typename elem_of<DT>::type v) {
    if constexpr (DT == 2)
        return v;
    else
        return from_bits<DT>(v);
}
template <int DT>
__device__ __forceinline__ typename elem_of<DT>::type f32_elem(float v) {
    if constexpr (DT == 2)
        return v;
    else
        return to_bits<DT>(v);
}

// 16 bytes of elements as fp32 (8 of 16-bit types, 4 of fp32)
template <int DT> constexpr int kVec = DT == 2 ? 4 : 8;
template <int DT>
__device__ __forceinline__ void unpack16(u32x4_t v, float* f) {
    if constexpr (DT == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == 0) {
                f[2 * i] = __uint_as_float(v[i] << 16);
                f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
            } else {
                f[2 * i] = f16_bits_to_f32((uint16_t)v[i]);
                f[2 * i + 1] = f16_bits_to_f32((uint16_t)(v[i] >> 16));
            }
        }
    }
}

// Monotone map of a float to uint32: a < b as values <=> key(a) < key(b); -0
// and +0 share a key, every NaN has the largest one.  0 is no float's key.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
    if (x != x) return 0xffffffffu;
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
// the same for values that are no NaN (a NaN gets some key)
__device__ __forceinline__ uint32_t order_key_finite(float x) {
    const int u = (int)__float_as_uint(x + 0.0f);
    return (uint32_t)(u ^ ((u >> 31) | (int)0x80000000));
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);  // the NaN key gives a NaN
}
// value and index in one: larger value first, then the lower index
__device__ __forceinline__ uint64_t order_key64(uint32_t key, uint32_t idx) {
    return ((uint64_t)key << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ uint32_t key64_index(uint64_t k) { return ~(uint32_t)k; }

template <typename T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const T o = __shfl_xor(v, d, 64);
        v = o > v ? o : v;
    }
    return v;
}

// Sum and maximum over a wave with DPP row shifts and broadcasts: six VALU
// steps, where a shuffle is an LDS round trip each (routing one token through
// 8 selections: ~0.4 us against ~1.5 us).  All 64 lanes must be active; the
// result is in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t old, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, dpp_u32<0x111, 0xf>(v, v));  // row_shr:1, 2, 4, 8
    v = max(v, dpp_u32<0x112, 0xf>(v, v));
    v = max(v, dpp_u32<0x114, 0xf>(v, v));
    v = max(v, dpp_u32<0x118, 0xf>(v, v));
    v = max(v, dpp_u32<0x142, 0xa>(v, v));  // row_bcast:15
    v = max(v, dpp_u32<0x143, 0xc>(v, v));  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __uint_as_float(dpp_u32<CTRL, ROWS>(0u, __float_as_uint(v)));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0x111, 0xf>(v);
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);
    v = dpp_add<0x143, 0xc>(v);
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Over 16 neighbouring lanes (row_ror: 8, 4, 2, 1), the result in each of them
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, dpp_u32<0x128, 0xf>(v, v));
    v = max(v, dpp_u32<0x124, 0xf>(v, v));
    v = max(v, dpp_u32<0x122, 0xf>(v, v));
    return max(v, dpp_u32<0x121, 0xf>(v, v));
}
__device__ __forceinline__ float row16_sum(float v) {
    v = dpp_add<0x128, 0xf>(v);
    v = dpp_add<0x124, 0xf>(v);
    v = dpp_add<0x122, 0xf>(v);
    return dpp_add<0x121, 0xf>(v);
}

}  // namespace omm

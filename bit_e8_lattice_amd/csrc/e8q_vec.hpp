// 16-byte vectors of float32 and bfloat16 values, and conversions, for the
// operators around the projection.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace e8q {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <typename T>
inline constexpr int kVec = int(16 / sizeof(T));   // elements per 16-byte vector (T: float, or uint16_t for bf16)

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

// Nearest even, NaN stays a NaN (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    const f32x2_t f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) { return uint16_t(cvt_bf16x2(v, 0.0f)); }

__device__ __forceinline__ void unpack(const u32x4_t& r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void unpack(const u32x4_t& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ u32x4_t pack(const float (&v)[4]) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]);
    return r;
}
__device__ __forceinline__ u32x4_t pack(const float (&v)[8]) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
    return r;
}

// Value of the lane whose number differs by the bits of MASK (a power of two),
// by register moves between lanes (no LDS).
template <int MASK>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
    if constexpr (MASK == 1) return uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, true));        // quad 1 0 3 2
    else if constexpr (MASK == 2) return uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, true));   // quad 2 3 0 1
    else if constexpr (MASK == 4) {                                                // mirror of 8 (^ 7), quad 3 2 1 0 (^ 3)
        const int m = __builtin_amdgcn_mov_dpp(int(v), 0x141, 0xF, 0xF, true);
        return uint32_t(__builtin_amdgcn_mov_dpp(m, 0x1B, 0xF, 0xF, true));
    } else if constexpr (MASK == 8) {
        return uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x128, 0xF, 0xF, true));  // rotate 16 by 8
    } else if constexpr (MASK == 16) {
        // rows 1 and 3 of the first result, 0 and 2 of the second come from their partner
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return (__lane_id() & 16u) ? r[0] : r[1];
    } else {
        static_assert(MASK == 32, "a power of two below 64");
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (__lane_id() & 32u) ? r[0] : r[1];
    }
}

template <int MASK>
__device__ __forceinline__ float lane_xor(float v) {
    return __uint_as_float(lane_xor<MASK>(__float_as_uint(v)));
}

template <int MASK>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v) {
    return (uint64_t(lane_xor<MASK>(uint32_t(v >> 32))) << 32) | lane_xor<MASK>(uint32_t(v));
}

}  // namespace e8q

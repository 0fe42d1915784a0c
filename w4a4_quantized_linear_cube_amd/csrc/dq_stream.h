// Rows of a stream (bf16 or fp32) in registers, 8 channels a lane: loads and
// stores, MX-FP8 codes, and fp64 sums over lanes in a fixed order.
#pragma once

#include "dq_device.h"

namespace dq {

typedef uint32_t v4w __attribute__((ext_vector_type(4)));
typedef uint32_t v2w __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v4w get16(const void* p) { return *(const v4w*)p; }
template <bool NT, class V>
__device__ __forceinline__ void put(void* p, V v) {
    if constexpr (NT) __builtin_nontemporal_store(v, (V*)p);
    else *(V*)p = v;
}

template <class T> struct Stream;
template <> struct Stream<uint16_t> {
    // 8 channels as they are loaded, and their values: for code that has more to load before it uses them
    typedef v4w Raw;
    static __device__ __forceinline__ Raw raw(const uint16_t* p) { return get16(p); }
    static __device__ __forceinline__ void values(Raw w, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void load(const uint16_t* p, float* v) {
        const v4w w = get16(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ float round(float v) { return (float)(__bf16)v; }
    template <bool NT> static __device__ __forceinline__ void store(uint16_t* p, const float* v) {
        v8bf b;
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = (__bf16)v[i];
        put<NT>(p, __builtin_bit_cast(v4w, b));
    }
};
template <> struct Stream<float> {
    struct Raw {
        v4w a, b;
    };
    static __device__ __forceinline__ Raw raw(const float* p) { return {get16(p), get16(p + 4)}; }
    static __device__ __forceinline__ void values(Raw w, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(w.a[i]);
            v[4 + i] = __uint_as_float(w.b[i]);
        }
    }
    static __device__ __forceinline__ void load(const float* p, float* v) {
        const v4w a = get16(p), b = get16(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(a[i]);
            v[4 + i] = __uint_as_float(b[i]);
        }
    }
    static __device__ __forceinline__ float round(float v) { return v; }
    template <bool NT> static __device__ __forceinline__ void store(float* p, const float* v) {
        put<NT>(p, v4f{v[0], v[1], v[2], v[3]});
        put<NT>(p + 4, v4f{v[4], v[5], v[6], v[7]});
    }
};

// Codes of 8 consecutive values, each v / scale rounded to nearest even.
__device__ __forceinline__ v2w encode8(const float* v, float scale) {
    v2s z = {0, 0};
    v2s a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, v[0], v[1], scale, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[2], v[3], scale, true);
    v2s b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, v[4], v[5], scale, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[6], v[7], scale, true);
    return v2w{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}

// Sums over lanes, pairwise by the bits of a lane's place, lowest first.
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
    const v2w w = __builtin_bit_cast(v2w, v);
    return __builtin_bit_cast(double, v2w{(uint32_t)__builtin_amdgcn_mov_dpp((int)w[0], CTRL, 0xF, 0xF, true),
                                          (uint32_t)__builtin_amdgcn_mov_dpp((int)w[1], CTRL, 0xF, 0xF, true)});
}
// ... of the lane 16 (32) places on, for the lower of two rows (halves); both get the sum
__device__ __forceinline__ double add_row(double v) {
    const v2w w = __builtin_bit_cast(v2w, v);
    const v2w lo = __builtin_amdgcn_permlane16_swap(w[0], w[0], false, false), hi = __builtin_amdgcn_permlane16_swap(w[1], w[1], false, false);
    return __builtin_bit_cast(double, v2w{lo[0], hi[0]}) + __builtin_bit_cast(double, v2w{lo[1], hi[1]});
}
__device__ __forceinline__ double add_half(double v) {
    const v2w w = __builtin_bit_cast(v2w, v);
    const v2w lo = __builtin_amdgcn_permlane32_swap(w[0], w[0], false, false), hi = __builtin_amdgcn_permlane32_swap(w[1], w[1], false, false);
    return __builtin_bit_cast(double, v2w{lo[0], hi[0]}) + __builtin_bit_cast(double, v2w{lo[1], hi[1]});
}
__device__ __forceinline__ double first_lane(double v) {
    const v2w w = __builtin_bit_cast(v2w, v);
    return __builtin_bit_cast(double, v2w{(uint32_t)__builtin_amdgcn_readfirstlane((int)w[0]), (uint32_t)__builtin_amdgcn_readfirstlane((int)w[1])});
}
// The sum of each N neighbouring lanes, in all of them.  (The lanes of a group
// of 4 hold one sum already, so a mirrored half row serves for the lane 4
// places on, and a mirrored row for that 8 places on.)
template <int N>
__device__ __forceinline__ double sum_lanes(double v) {
    if constexpr (N > 1) v += moved<0xB1>(v);          // lane ^ 1
    if constexpr (N > 2) v += moved<0x4E>(v);          // lane ^ 2
    if constexpr (N > 4) v += moved<0x141>(v);
    if constexpr (N > 8) v += moved<0x140>(v);
    if constexpr (N > 16) v = add_row(v);
    if constexpr (N > 32) v = add_half(v);
    return v;
}

}  // namespace dq

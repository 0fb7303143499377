// Element types of the operators around a projection (norms, adapters):
// fp32, fp16 or bf16 arrays chosen by a run-time type code.  Loads are split
// from conversions, so that a thread can have all of its loads in flight
// before the first conversion waits for one.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/pq2.h"

namespace pq2 {

// V consecutive elements as loaded: V = 8 (32 bytes of fp32, 16 of a 16-bit
// type) or V = 1.
template <int V>
struct RawVec;
template <>
struct RawVec<8> {
    uint4 a, b;
};
template <>
struct RawVec<1> {
    uint32_t a;
};

template <int V>
__device__ __forceinline__ RawVec<V> raw_zero() {
    if constexpr (V == 8)
        return {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    else
        return {0u};
}

// Elements i .. i + V - 1 of `base` (V = 8: base + i on a 16-byte boundary).
template <int V>
__device__ __forceinline__ RawVec<V> raw_load(const void* base, int type, size_t i) {
    RawVec<V> r = raw_zero<V>();
    if constexpr (V == 8) {
        if (type == PQ2_F32) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
            r.a = p[0];
            r.b = p[1];
        } else {
            r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
        }
    } else {
        if (type == PQ2_F32)
            r.a = static_cast<const uint32_t*>(base)[i];
        else
            r.a = static_cast<const uint16_t*>(base)[i];
    }
    return r;
}

__device__ __forceinline__ float elem_to_f32(uint32_t bits16, int type) {
    if (type == PQ2_BF16) return __uint_as_float(bits16 << 16);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits16)));
}

template <int V>
__device__ __forceinline__ void raw_to_f32(const RawVec<V>& r, int type, float (&v)[V]) {
    if constexpr (V == 8) {
        const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
        if (type == PQ2_F32) {
            const uint32_t b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = __uint_as_float(a[j]);
                v[4 + j] = __uint_as_float(b[j]);
            }
        } else if (type == PQ2_BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(a[j] << 16);
                v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[j]));
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        }
    } else {
        v[0] = type == PQ2_F32 ? __uint_as_float(r.a) : elem_to_f32(r.a, type);
    }
}

// One rounding to nearest even of each value to the array's type.
__device__ __forceinline__ uint16_t f32_to_elem16(float v, int type) {
    if (type == PQ2_BF16) {
        const __nv_bfloat16 b = __float2bfloat16_rn(v);
        return *reinterpret_cast<const uint16_t*>(&b);
    }
    return __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ uint32_t f32x2_to_elem16(float lo, float hi, int type) {
    if (type == PQ2_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <int V>
__device__ __forceinline__ void store_f32(void* base, int type, size_t i, const float (&v)[V]) {
    if constexpr (V == 8) {
        if (type == PQ2_F32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
                make_uint4(f32x2_to_elem16(v[0], v[1], type), f32x2_to_elem16(v[2], v[3], type),
                           f32x2_to_elem16(v[4], v[5], type), f32x2_to_elem16(v[6], v[7], type));
        }
    } else {
        if (type == PQ2_F32)
            static_cast<float*>(base)[i] = v[0];
        else
            static_cast<uint16_t*>(base)[i] = f32_to_elem16(v[0], type);
    }
}

}  // namespace pq2

// vecio.cuh -- V consecutive elements as one register-packed access (16 bytes)
// or a single element, converted to and from fp32.
#pragma once

#include "common.cuh"

namespace gdn {

// Raw stays in 32-bit registers until it is unpacked: an array of 16-bit
// elements would take a register each.
template <typename T, int V> struct Pack;
template <> struct Pack<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[4]) {
        x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
    }
    static __device__ __forceinline__ Raw pack(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
    static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <> struct Pack<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[8]) {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
};
template <typename T> struct Pack<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[1]) { x[0] = to_f32(r); }
    static __device__ __forceinline__ Raw pack(const float (&x)[1]) { return from_f32<T>(x[0]); }
    static __device__ __forceinline__ Raw zero() { return from_f32<T>(0.f); }
};

}  // namespace gdn

// values.cuh -- reading and writing tensors of float, bf16 and fp16 values, 16 bytes at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ep_internal.cuh"

namespace ep {

template <typename V>
struct Io;
template <>
struct Io<float> {
    static constexpr int kVec = 4;
    static __device__ float load(const float *p) { return *p; }
    static __device__ void store(float *p, float v) { *p = v; }
    static __device__ void unpack(const uint4 &q, float (&v)[4]) {
        v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
    }
    static __device__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct Io<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static __device__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ void store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
    static __device__ void unpack(const uint4 &q, float (&v)[8]) {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    static __device__ uint4 pack(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Io<__half> {
    static constexpr int kVec = 8;
    static __device__ float load(const __half *p) { return __half2float(*p); }
    static __device__ void store(__half *p, float v) { *p = __float2half_rn(v); }
    static __device__ void unpack(const uint4 &q, float (&v)[8]) {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
    static __device__ uint4 pack(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// Values before the first 16-byte boundary at or after p.
template <typename V>
__device__ __forceinline__ int64_t values_to_boundary(const V *p) {
    return (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(V);
}

}  // namespace ep

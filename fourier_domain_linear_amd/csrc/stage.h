// stage.h -- element access shared by the norm and rotary kernels: vectors of 16 bytes as fp32 values.
#pragma once

#include "device_common.h"
#include "eqlin_internal.h"

namespace eqlin {

struct F32 {};  // element tag of the fp32 kernels

template <class E>
struct Elem {
    typedef uint16_t T;
    static constexpr int V = 8;  // elements of a 16-byte vector
    static __device__ __forceinline__ float get(T x) { return elem_to_float<E>(x); }
    static __device__ __forceinline__ T put(float x) { return pack1<E>(x); }
    static __device__ __forceinline__ void unpack(const uint4 &u, float *f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = elem_at<E>(u, j);
    }
    static __device__ __forceinline__ uint4 pack(const float *f) { return pack8<E>(f); }
};
template <>
struct Elem<F32> {
    typedef float T;
    static constexpr int V = 4;
    static __device__ __forceinline__ float get(T x) { return x; }
    static __device__ __forceinline__ T put(float x) { return x; }
    static __device__ __forceinline__ void unpack(const uint4 &u, float *f) {
        f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
    return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
    return x;
}

}  // namespace eqlin

// stage.h -- element access shared by the norm, rotary and recurrence kernels: vectors as fp32 values.
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

// W elements (16, 8, 4 bytes or a single half), loaded and stored at once; pointers aligned to them.
template <class E, int W>
struct Pack {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    static constexpr int kWords = W * (int)sizeof(T) / 4;  // 0: a single half
    uint32_t w[kWords ? kWords : 1];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < (kWords ? kWords : 1); ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kWords == 4) {
            const uint4 u = *(const uint4 *)p;
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else if constexpr (kWords == 2) {
            const uint2 u = *(const uint2 *)p;
            w[0] = u.x, w[1] = u.y;
        } else if constexpr (kWords == 1) {
            w[0] = *(const uint32_t *)p;
        } else {
            static_assert(W == 1, "16, 8, 4 bytes or one element");
            w[0] = *(const uint16_t *)p;
        }
    }
    __device__ __forceinline__ void unpack(float *f) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < W; ++j) f[j] = __uint_as_float(w[j]);
        } else if constexpr (W == 1) {
            f[0] = EL::get((T)w[0]);
        } else {
#pragma unroll
            for (int j = 0; j < W; j += 2) f[j] = elem_lo<E>(w[j / 2]), f[j + 1] = elem_hi<E>(w[j / 2]);
        }
    }
    static __device__ __forceinline__ void store(T *p, const float *f) {
        if constexpr (kWords == 4) *(uint4 *)p = EL::pack(f);
        else if constexpr (sizeof(T) == 4 && W == 2) *(uint2 *)p = make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1]));
        else if constexpr (W == 4) *(uint2 *)p = make_uint2(pack2<E>(f[0], f[1]), pack2<E>(f[2], f[3]));
        else if constexpr (W == 2) *(uint32_t *)p = pack2<E>(f[0], f[1]);
        else *p = EL::put(f[0]);
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

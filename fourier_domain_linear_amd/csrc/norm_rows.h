// norm_rows.h -- what the norm kernels share: sums over the lanes of a row, launch sizes.
#pragma once

#include "stage.h"

namespace eqlin {

// Sum over the lanes that share a row: a wave, or the whole workgroup (through LDS).
template <int WAVES>
struct RowGroup {
    float *red;
    __device__ __forceinline__ float sum(float x) {
        x = wave_sum(x);
        if constexpr (WAVES > 1) {
            __syncthreads();
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
            __syncthreads();
            x = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) x += red[w];
        }
        return x;
    }
    __device__ __forceinline__ float max(float x) {
        x = wave_max(x);
        if constexpr (WAVES > 1) {
            __syncthreads();
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
            __syncthreads();
            x = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) x = fmaxf(x, red[w]);
        }
        return x;
    }
};

// workgroups for `rows`, rows_per_wg at a time, at most per_cu a compute unit
inline unsigned grid_for(int64_t rows, int rows_per_wg, int per_cu) {
    const int64_t need = (rows + rows_per_wg - 1) / rows_per_wg, most = (int64_t)device_num_cus() * per_cu;
    return (unsigned)std::max<int64_t>(1, std::min(need, most));
}

}  // namespace eqlin

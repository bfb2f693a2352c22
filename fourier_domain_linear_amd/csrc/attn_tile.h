// attn_tile.h -- tiles of keys and values through LDS, shared by the forward and the dQ kernel.
#pragma once

#include "attn.h"

namespace eqlin {

// 4 waves, each 32 packed rows (the columns of S^T), all over the same key tiles.
template <class E, int DP>
struct TileCfg {
    typedef Tile<E, DP> TL;
    static constexpr int kWaves = 4;
    static constexpr int BM = 32 * kWaves;                     // packed rows of a workgroup
    static constexpr int NKB = __is_same(E, F32) ? 1 : 2;      // 32-key blocks of a tile
    static constexpr int BN = 32 * NKB;
    static constexpr int kTileBytes = BN * TL::kRow;
    static constexpr int kLds = 4 * kTileBytes;                // k and v, two buffers
    static constexpr int kStage = kTileBytes / 16 / (64 * kWaves);  // 16-byte chunks a thread stages per tile
    static_assert(kTileBytes % (16 * 64 * kWaves) == 0, "whole chunks");
};

// One tile of `rows` x D elements (row stride in elements) from global memory, in 16-byte chunks; rows from
// `valid` on and columns from D on read as zero.
template <class E, int DP, int N, int THREADS>
struct Stage {
    typedef Tile<E, DP> TL;
    typedef typename ElemOf<E>::type T;
    uint4 r[N];
    __device__ __forceinline__ void load(const T *base, int64_t stride, int valid, int D, int tid) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int id = tid + j * THREADS, row = id / TL::kChunks, c = id % TL::kChunks;
            const int col = c * (16 / (int)sizeof(T));
            r[j] = row < valid && col < D ? *(const uint4 *)(base + row * stride + col) : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void store(char *tile, int tid) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int id = tid + j * THREADS, row = id / TL::kChunks, c = id % TL::kChunks;
            *(uint4 *)(tile + TL::at(row, c)) = r[j];
        }
    }
};

// Stores a column's 32 db + d_row(v, h) values (o^T in D layout), scaled, to dst[0..D).
template <class E, int DP>
__device__ __forceinline__ void store_column(const f32x16 *o, float inv, typename ElemOf<E>::type *dst, int D, int h) {
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int d = 32 * db + 8 * g + 4 * h;
            if (d < D) {
                if constexpr (__is_same(E, F32))
                    *(float4 *)(dst + d) = make_float4(o[db][4 * g] * inv, o[db][4 * g + 1] * inv, o[db][4 * g + 2] * inv,
                                                       o[db][4 * g + 3] * inv);
                else
                    *(uint2 *)(dst + d) = make_uint2(pack2<E>(o[db][4 * g] * inv, o[db][4 * g + 1] * inv),
                                                     pack2<E>(o[db][4 * g + 2] * inv, o[db][4 * g + 3] * inv));
            }
        }
}

}  // namespace eqlin

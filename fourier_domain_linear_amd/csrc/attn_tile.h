// attn_tile.h -- tiles of keys, values or packed query rows from global memory into LDS, and the stores of
// results, shared by the attention kernels.
#pragma once

#include "attn.h"

// m0 is written and used inside one asm statement
#pragma clang diagnostic ignored "-Winline-asm"

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
    static constexpr int kFlags = 2 * 4 * 4;                   // a word a wave, two sets
};

// Units an XCD takes in a run: the tiles of a sequence where they are few, else one.
inline int run_of(int64_t slots, int B) { return slots > 16 * (int64_t)B ? 1 : (int)std::max<int64_t>(1, (slots + B - 1) / B); }

// LDS offset (bytes) of a pointer into the workgroup's LDS.
__device__ __forceinline__ uint32_t lds_offset(const char *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// 1 KB from global memory straight into LDS: lane l's 16 bytes at base + off go to lds + 16 l. The compiler does
// not see these loads (it would wait for them before every later LDS read): dma_wait() before the barrier that
// publishes them. The wait states are those of a scalar base that a vector instruction has just written, which the
// compiler cannot count inside asm.
__device__ __forceinline__ void dma_1k(uint32_t lds, const void *base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// All but the youngest N loads of the wave (they arrive in order).
template <int N>
__device__ __forceinline__ void dma_wait_but() {
    static_assert(N < 64, "six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The wave's LDS reads so far have their values.
__device__ __forceinline__ void lds_read_wait() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A tile of ROWS rows, moved by the workgroup's WAVES waves. Chunks are permuted on the way (a lane fetches the
// chunk that the swizzle puts at its place). Rows past the last valid one repeat it; columns from D on are
// not written (zero_pad clears them once).
template <class E, int DP, int ROWS, int WAVES = 4>
struct TileDma {
    typedef Tile<E, DP> TL;
    typedef typename ElemOf<E>::type T;
    static constexpr int N = ROWS * TL::kRow / (1024 * WAVES);
    static_assert(ROWS * TL::kRow % (1024 * WAVES) == 0, "whole kilobytes");
    uint32_t off[N];
    __device__ static __forceinline__ int place(int wave, int lane, int j) { return (j * WAVES + wave) * 1024 + lane * 16; }
    __device__ static __forceinline__ int row_of(int wave, int lane, int j) { return place(wave, lane, j) / TL::kRow; }
    __device__ static __forceinline__ int col_of(int wave, int lane, int j) {  // first element of the chunk
        const int at = place(wave, lane, j);
        return (((at % TL::kRow) >> 4) ^ TL::swz(at / TL::kRow)) * (16 / (int)sizeof(T));
    }
    // rows of one stride, `valid` of them (> 0)
    __device__ __forceinline__ void offsets(int64_t stride, int valid, int wave, int lane) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            off[j] = ((uint32_t)min(row_of(wave, lane, j), valid - 1) * (uint32_t)stride + (uint32_t)col_of(wave, lane, j)) * (uint32_t)sizeof(T);
    }
    // packed rows: row `rem` + r of the tokens from the base on, head (rem + r) % grp
    __device__ __forceinline__ void offsets_packed(int64_t ts, int64_t hs, int rem, int grp, int valid, int wave, int lane) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t r = (uint32_t)(rem + min(row_of(wave, lane, j), valid - 1)), t = r / (uint32_t)grp, h = r - t * (uint32_t)grp;
            off[j] = (t * (uint32_t)ts + h * (uint32_t)hs + (uint32_t)col_of(wave, lane, j)) * (uint32_t)sizeof(T);
        }
    }
    __device__ __forceinline__ void issue(uint32_t lds, const T *tile, int D, int wave, int lane) const {
        const T *base = (const T *)uniform((int64_t)tile);  // into scalar registers
        if (D == DP) {
#pragma unroll
            for (int j = 0; j < N; ++j) dma_1k(lds + (j * WAVES + wave) * 1024, base, off[j]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (col_of(wave, lane, j) < D) dma_1k(lds + (j * WAVES + wave) * 1024, base, off[j]);
        }
    }
};

// Clears LDS where heads are padded to DP: the columns from D on stay zero.
template <int THREADS = 256>
__device__ __forceinline__ void zero_pad(char *lds, int bytes, int D, int DP, int tid) {
    if (D == DP) return;
    for (int i = tid * 16; i < bytes; i += THREADS * 16) *(uint4 *)(lds + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
}

// Stores a column's 32 db + d_row(v, h) values (o^T in D layout), scaled, to dst[0..D), 16 bytes a lane: lanes l and
// l ^ 32 hold neighbouring fours of the same row and exchange them, so that each has eight in a row.
template <class E, int DP>
__device__ __forceinline__ void store_column(const f32x16 *o, float inv, typename ElemOf<E>::type *dst, int D, int h) {
#pragma unroll
    for (int db = 0; db < DP / 32; ++db) {
        if constexpr (__is_same(E, F32)) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int d = 32 * db + 8 * g + 4 * h;
                if (d < D)
                    *(float4 *)(dst + d) = make_float4(o[db][4 * g] * inv, o[db][4 * g + 1] * inv, o[db][4 * g + 2] * inv,
                                                       o[db][4 * g + 3] * inv);
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                uint32_t a[2], b[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int v = 4 * g + 2 * j;
                    const auto r = __builtin_amdgcn_permlane32_swap(pack2<E>(o[db][v] * inv, o[db][v + 1] * inv),
                                                                    pack2<E>(o[db][v + 4] * inv, o[db][v + 5] * inv), false, false);
                    a[j] = r[0], b[j] = r[1];
                }
                const int d = 32 * db + 8 * g + 8 * h;
                if (d < D) *(uint4 *)(dst + d) = make_uint4(a[0], a[1], b[0], b[1]);
            }
        }
    }
}

// The B-operand fragments of a lane's row (dims in 16-byte chunks, zeros from D on).
template <class E, int DP>
__device__ __forceinline__ void load_row(uint4 *f, const typename ElemOf<E>::type *row, int D, int h) {
    constexpr int kPer = 16 / (int)sizeof(typename ElemOf<E>::type);
    if (D == DP) {
#pragma unroll
        for (int t = 0; t < Tile<E, DP>::kSteps; ++t) f[t] = *(const uint4 *)(row + (2 * t + h) * kPer);
    } else {
#pragma unroll
        for (int t = 0; t < Tile<E, DP>::kSteps; ++t)
            f[t] = (2 * t + h) * kPer < D ? *(const uint4 *)(row + (2 * t + h) * kPer) : make_uint4(0, 0, 0, 0);
    }
}

// ---- values of tokens that a row must not see ----
//
// A masked probability is 0, but the second product multiplies it with whatever the masked token holds, and 0 times
// an infinity or NaN is NaN. Tiles that some row sees only in part are therefore looked over, and where one holds such
// a value, the tile's place is cleared and the rows that do see it get it added at the end (finite everywhere
// else: the products are unchanged). A tile is looked over once or twice a workgroup; the rest never runs in ordinary use.

template <class E>
__device__ __forceinline__ uint32_t nonfinite_mask(uint32_t w) {  // the bits of the word's values that are not finite
    if constexpr (__is_same(E, F32)) {
        return (w & 0x7f800000u) == 0x7f800000u ? 0xffffffffu : 0u;
    } else {
        constexpr uint32_t e = __is_same(E, F16) ? 0x7c00u : 0x7f80u;
        return ((w & e) == e ? 0xffffu : 0u) | ((w & (e << 16)) == (e << 16) ? 0xffff0000u : 0u);
    }
}
// Whether this thread's share of a tile holds such a value.
template <class E, int THREADS>
__device__ __forceinline__ bool tile_nonfinite(const char *tile, int bytes, int tid) {
    uint32_t any = 0;
#pragma unroll 1
    for (int i = tid * 16; i < bytes; i += THREADS * 16) {
        const uint4 v = *(const uint4 *)(tile + i);
        any |= nonfinite_mask<E>(v.x) | nonfinite_mask<E>(v.y) | nonfinite_mask<E>(v.z) | nonfinite_mask<E>(v.w);
    }
    return any != 0;
}
template <class E, int THREADS>
__device__ __forceinline__ void clear_nonfinite(char *tile, int bytes, int tid) {
#pragma unroll 1
    for (int i = tid * 16; i < bytes; i += THREADS * 16) {
        uint4 v = *(const uint4 *)(tile + i);
        v.x &= ~nonfinite_mask<E>(v.x), v.y &= ~nonfinite_mask<E>(v.y), v.z &= ~nonfinite_mask<E>(v.z), v.w &= ~nonfinite_mask<E>(v.w);
        *(uint4 *)(tile + i) = v;
    }
}
// After the tiles: acc[d] += X[r][d] for the rows r of [from, to] that the lane's column sees and the values that are
// not finite, from global memory (row(r): the row's first element).
template <class E, int DP, class Row, class Sees>
__device__ __forceinline__ void add_nonfinite(f32x16 *acc, int from, int to, int D, int h, Row row, Sees sees) {
    typedef typename ElemOf<E>::type T;
#pragma unroll 1
    for (int r = from; r <= to; ++r) {
        const bool see = sees(r);
        const T *x = row(r);
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int d = 32 * db + 8 * g + 4 * h;
                if (d < D)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v = Elem<E>::get(x[d + j]);
                        acc[db][4 * g + j] += see && !(fabsf(v) < INFINITY) ? v : 0.0f;
                    }
            }
    }
}

// The same for a tile that also made the scores: a column that sees a row with such a value becomes NaN whole.
template <class E, int DP, class Row, class Sees>
__device__ __forceinline__ void poison_columns(f32x16 *acc, int from, int to, int D, int h, Row row, Sees sees) {
    typedef typename ElemOf<E>::type T;
    float add = 0.0f;
#pragma unroll 1
    for (int r = from; r <= to; ++r) {
        const T *x = row(r);
        bool bad = false;
        for (int d = h; d < D; d += 2) bad |= !(fabsf(Elem<E>::get(x[d])) < INFINITY);
        bad = (__ballot(bad) & (1ull | 1ull << 32)) != 0;  // the row's two halves of values, the same for every lane
        if (bad && sees(r)) add = NAN;
    }
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[db][v] += add;
}

}  // namespace eqlin

// attn.h -- what the attention kernels share: parameters, the sequence of a tile, operand fragments.
//
// Rows. The query heads that share a key-value head ("a group") are rows of one product: packed row
// r = token * group + head-in-group, so a key tile is read once for the whole group and a step of one new
// token still fills matrix-core columns.
//
// Products. S^T = K Q^T is computed with keys as rows and queries as columns (D of a 32x32 product: lane l
// holds column l % 32 and rows 8 (v / 4) + 4 (l / 32) + v % 4). The softmax statistics of a query are then
// one lane's (and its partner's, l ^ 32), and the probabilities a lane holds are already the B operand of
// O^T = V^T P^T when the 16 (half types) reduction slots of a step are taken in the order the lane has them:
// slot 8 h + j is key 16 s + 4 h + (j % 4) + 8 (j / 4) of step s (h = l / 32). V^T is read from the
// row-major tile with the LDS transpose read in that key order. The backward's products follow the same rule.
#pragma once

#include "stage.h"
#include "eqlin_internal.h"

namespace eqlin {



template <class E>
struct ElemOf {
    typedef uint16_t type;
};
template <>
struct ElemOf<F32> {
    typedef float type;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---- fragments: one uint4 a lane = half of a step's reduction slots (half types: 16 slots a step, one
// 32x32x16 product; fp32: 8 slots, four 32x32x2 products) ----

template <class E>
__device__ __forceinline__ f32x16 mma_frag(const uint4 &a, const uint4 &b, f32x16 c) {
    if constexpr (__is_same(E, F32)) {
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
        return c;
    } else {
        return mma32<E>(a, b, c);
    }
}

// W (a 32x32 product's D layout, 16 values a lane) -> B-operand fragments of the next product: NF = 2
// (half types, rounded to nearest even) or 4 (fp32, exact).
template <class E>
struct WFrags {
    static constexpr int NF = __is_same(E, F32) ? 4 : 2;
    uint4 f[NF];
    __device__ __forceinline__ void set(const f32x16 &w) {
        if constexpr (__is_same(E, F32)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = make_uint4(__float_as_uint(w[4 * i]), __float_as_uint(w[4 * i + 1]), __float_as_uint(w[4 * i + 2]),
                                  __float_as_uint(w[4 * i + 3]));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float t[8] = {w[8 * i],     w[8 * i + 1], w[8 * i + 2], w[8 * i + 3],
                                    w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]};
                f[i] = pack8<E>(t);
            }
        }
    }
};

// ---- LDS tiles: [rows][DP] of the element type, 16-byte chunks XOR-swizzled by the row so that both the
// row reads (16 consecutive rows, one chunk) and the transpose reads (4 consecutive rows, 64 bytes of each)
// spread over all banks ----

template <class E, int DP>
struct Tile {
    typedef typename ElemOf<E>::type T;
    static constexpr int kRow = DP * (int)sizeof(T);  // bytes
    static constexpr int kChunks = kRow / 16;
    static constexpr int kSteps = kChunks / 2;  // steps of a product that reduces over d

    __device__ static __forceinline__ int swz(int row) {
        if constexpr (kRow >= 256) return ((row & 3) << 2) | ((row >> 2) & 3);
        else if constexpr (kRow == 128) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
        else return (row >> 2) & 3;
    }
    __device__ static __forceinline__ int at(int row, int chunk) { return row * kRow + ((chunk ^ swz(row)) << 4); }

    // A (or B) operand of a product reducing over d: row `row` of the tile, step s
    __device__ static __forceinline__ uint4 row_frag(const char *tile, int row, int s, int h) {
        return *(const uint4 *)(tile + at(row, 2 * s + h));
    }
    // A operand of a product reducing over the tile's rows: rows (of the product) d = 32 db + lane % 32,
    // reduction slots = tile rows row0 + the D-layout rows of W's fragment f (32 rows from row0)
    __device__ static __forceinline__ uint4 col_frag(const char *tile, int row0, int f, int db, int lane) {
        const int h = lane >> 5;
        if constexpr (__is_same(E, F32)) {
            uint4 r;
            uint32_t v[4];
            const int d = 32 * db + (lane & 31);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = row0 + 8 * f + 4 * h + j;
                v[j] = *(const uint32_t *)(tile + at(row, d >> 2) + (d & 3) * 4);
            }
            r.x = v[0], r.y = v[1], r.z = v[2], r.w = v[3];
            return r;
        } else {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
            const int l16 = lane & 15;
            const int row = row0 + 16 * f + 4 * h + (l16 >> 2);
            const int chunk = 4 * db + 2 * ((lane >> 4) & 1) + ((l16 >> 1) & 1);
            const char *p0 = tile + at(row, chunk) + (l16 & 1) * 8;
            const char *p1 = tile + at(row + 8, chunk) + (l16 & 1) * 8;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p0);
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p1);
            const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
            return make_uint4(ua.x, ua.y, ub.x, ub.y);
        }
    }
};

// ---- lanes ----

// {own value, partner's} of lanes l and l ^ 32 as {value of the low lane, value of the high lane}
__device__ __forceinline__ void halves(float x, float &lo, float &hi) {
    const uint32_t u = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    lo = __uint_as_float(r[0]);
    hi = __uint_as_float(r[1]);
}
__device__ __forceinline__ float half_max(float x) {
    float a, b;
    halves(x, a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float half_sum(float x) {
    float a, b;
    halves(x, a, b);
    return a + b;
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// D-layout row of value v for lane half h
__device__ __forceinline__ constexpr int d_row(int v, int h) { return (v & 3) + 8 * (v >> 2) + 4 * h; }

// ---- sequences ----

struct Seq {
    int64_t q0, k0;  // first packed query token and key
    int lq, lk;      // tokens; keys that count
    int lk_slot;     // keys of the packed slot (>= lk)
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

// Sequence i, with every bound forced into the tensors whatever the arrays hold.
__device__ __forceinline__ Seq seq_at(const AttnParams &p, int i) {
    Seq s;
    s.q0 = clamp64(p.cu_q[i], 0, p.total_q);
    s.lq = (int)(clamp64(p.cu_q[i + 1], s.q0, p.total_q) - s.q0);
    s.k0 = clamp64(p.cu_k[i], 0, p.total_k);
    s.lk_slot = (int)(clamp64(p.cu_k[i + 1], s.k0, p.total_k) - s.k0);
    s.lk = p.len_k ? (int)clamp64(p.len_k[i], 0, s.lk_slot) : s.lk_slot;
    return s;
}

// Tiles of `size` units over sequences of cu[i + 1] - cu[i] items of `mul` units: sequence i owns the tile
// slots from cu[i] * mul / size + i on, at least as many as it has tiles, so the launch needs no lengths on
// the host. Finds the sequence of a slot with a 64-way search by the wave, one load a level.
__device__ __forceinline__ int64_t slot_start(const int *cu, int i, int64_t total, int mul, int size) {
    return clamp64(cu[i], 0, total) * mul / size + i;
}
__device__ __forceinline__ int seq_of_slot(const int *cu, int B, int64_t total, int mul, int size, int64_t slot) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = B;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int i = lo + lane * step;
        const bool in = lane * step < n && slot_start(cu, i, total, mul, size) <= slot;
        int c = __popcll(__ballot(in));
        c = c < 1 ? 1 : c;
        const int skip = (c - 1) * step;
        lo += skip;
        n = n - skip < step ? n - skip : step;
    }
    return uniform(lo);
}

}  // namespace eqlin

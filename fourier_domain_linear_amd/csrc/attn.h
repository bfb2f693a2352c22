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

__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int v = 0; v < 16; ++v) z[v] = 0.0f;
    return z;
}

// W (a 32x32 product's D layout, 16 values a lane) -> B-operand fragments of the next product: NF = 2
// (half types, rounded to nearest even) or 4 (fp32, exact). The rounding is the price of the half types' products, seven
// times as fast as fp32's: o's error against 64 bits is 1.35 times that of o's own rounding alone.
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
    // Addresses. A tile begins at a multiple of 512 bytes and the swizzle takes the row modulo 16, so every
    // fragment's address is (tile + a lane's constant) XOR a compile-time constant, plus an immediate.
    struct Lane {
        uint32_t row, col0, col1;
    };
    __device__ static __forceinline__ Lane lane_of(int lane) {
        const int h = lane >> 5, l32 = lane & 31, l16 = lane & 15;
        Lane L;
        L.row = l32 * kRow + ((h ^ swz(l32)) << 4);
        if constexpr (__is_same(E, F32)) {
            L.col0 = 4 * h * kRow + (((l32 >> 2) ^ h) << 4) + (l32 & 3) * 4;
            L.col1 = 0;
        } else {
            const int r = 4 * h + (l16 >> 2), x = 2 * ((lane >> 4) & 1) + ((l16 >> 1) & 1);
            L.col0 = r * kRow + ((x ^ swz(r)) << 4) + (l16 & 1) * 8;
            L.col1 = (r + 8) * kRow + ((x ^ swz(r + 8)) << 4) + (l16 & 1) * 8;
        }
        return L;
    }
    template <class V>
    __device__ static __forceinline__ V lds_at(uint32_t a) {
        return *(const __attribute__((address_space(3))) V *)(uintptr_t)a;
    }
    // A (or B) operand of a product reducing over d: row 32 blk + lane % 32 of the tile, step s
    __device__ static __forceinline__ uint4 row_frag(uint32_t tile, const Lane &L, int blk, int s) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const u32x4 v = lds_at<u32x4>(((tile + L.row) ^ (s << 5)) + blk * 32 * kRow);
        return __builtin_bit_cast(uint4, v);
    }
    // A operand of a product reducing over the tile's rows: rows (of the product) d = 32 db + lane % 32,
    // reduction slots = the tile rows, from row 32 blk on, that W's fragment f holds
    __device__ static __forceinline__ uint4 col_frag(uint32_t tile, const Lane &L, int blk, int f, int db) {
        if constexpr (__is_same(E, F32)) {
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int sw = (kRow >= 256 ? j << 2 : (j >> 1) << 2) | (2 * (f & 1));
                v[j] = lds_at<uint32_t>(((tile + L.col0) ^ ((8 * db ^ sw) << 4)) + (32 * blk + 8 * f + j) * kRow);
            }
            return make_uint4(v[0], v[1], v[2], v[3]);
        } else {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
            const uint32_t at = (32 * blk + 16 * f) * kRow;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)(((tile + L.col0) ^ (db << 6)) + at));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)(((tile + L.col1) ^ (db << 6)) + at));
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
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32) | (uint32_t)uniform((int)x));
}

// D-layout row of value v for lane half h
__device__ __forceinline__ constexpr int d_row(int v, int h) { return (v & 3) + 8 * (v >> 2) + 4 * h; }

// Order of a block that multiplies LDS fragments: AHEAD reads first, then the others spread over the products, so
// that no product waits for its own read (left alone, the compiler reuses one register quad: read, wait, multiply).
template <int READS, int PRODUCTS, int AHEAD>
__device__ __forceinline__ void read_ahead() {
    constexpr int kRead = 0x100, kMfma = 0x8, kPer = READS / PRODUCTS;  // reads a product
    static_assert(READS % PRODUCTS == 0 && AHEAD % kPer == 0 && AHEAD <= READS, "whole products");
    __builtin_amdgcn_sched_group_barrier(kRead, AHEAD, 0);
#pragma unroll
    for (int i = 0; i < PRODUCTS - AHEAD / kPer; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kRead, kPer, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, AHEAD / kPer, 0);
}

// ---- sequences ----

struct Seq {
    int64_t q0, k0;  // first packed query token and key
    int lq, lk;      // tokens; keys that count
    int lk_slot;     // keys of the packed slot (>= lk)
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

// Tiles of `size` units over sequences of cu[i + 1] - cu[i] items of `mul` units: sequence i owns the tile
// slots from cu[i] * mul / size + i on, at least as many as it has tiles, so the launch needs no lengths on
// the host.
__device__ __forceinline__ int64_t slot_start(int64_t cu, int i, int mul, int size) { return cu * mul / size + i; }

// The last sequence i with before(i, cu[i]) (true up to it, false after), by a 64-way search of the wave. The last
// level's lanes load all that is asked of a sequence at once, so up to 64 sequences cost one round trip to memory.
// Every bound is forced into the tensors whatever the arrays hold. BY_K: cu is the keys', else the queries'.
template <bool BY_K, class Before>
__device__ __forceinline__ Seq find_seq(const AttnParams &p, Before before, int &index) {
    const int lane = threadIdx.x & 63;
    const int *cu = BY_K ? p.cu_k : p.cu_q;
    int lo = 0, n = p.B;
    while (n > 64) {
        const int step = (n + 63) / 64, i = lo + lane * step;
        const bool in = lane * step < n && before(i, cu[i < p.B ? i : p.B]);
        int c = __popcll(__ballot(in));
        c = c < 1 ? 1 : c;
        const int skip = (c - 1) * step;
        lo += skip;
        n = n - skip < step ? n - skip : step;
    }
    const int i = lo + (lane < n ? lane : n - 1);
    const int q0 = p.cu_q[i], q1 = p.cu_q[i + 1], k0 = p.cu_k[i], k1 = p.cu_k[i + 1], len = p.len_k ? p.len_k[i] : 0x7fffffff;
    const bool in = lane < n && before(i, BY_K ? k0 : q0);
    int c = __popcll(__ballot(in));
    c = uniform(c < 1 ? 0 : c - 1);
    index = uniform(lo) + c;
    auto clamp = [](int x, int a, int b) { return min(max(x, a), b); };
    const int q_at = clamp(__builtin_amdgcn_readlane(q0, c), 0, (int)p.total_q);
    const int k_at = clamp(__builtin_amdgcn_readlane(k0, c), 0, (int)p.total_k);
    Seq s;
    s.q0 = q_at, s.k0 = k_at;
    s.lq = clamp(__builtin_amdgcn_readlane(q1, c), q_at, (int)p.total_q) - q_at;
    s.lk_slot = clamp(__builtin_amdgcn_readlane(k1, c), k_at, (int)p.total_k) - k_at;
    s.lk = clamp(__builtin_amdgcn_readlane(len, c), 0, s.lk_slot);
    return s;
}

// The sequence of a slot and the slot's tile in it. BY_K: slots over the keys, else over the queries.
template <bool BY_K>
__device__ __forceinline__ Seq seq_of_slot(const AttnParams &p, int mul, int size, int64_t slot, int64_t &tile) {
    const int64_t total = BY_K ? p.total_k : p.total_q;
    int i;
    const Seq s = find_seq<BY_K>(p, [&](int j, int cu) { return slot_start(clamp64(cu, 0, total), j, mul, size) <= slot; }, i);
    tile = slot - slot_start(BY_K ? s.k0 : s.q0, i, mul, size);
    return s;
}

// The sequence of packed query token t (the last that begins at or before it).
__device__ __forceinline__ Seq seq_of_row(const AttnParams &p, int t, int &index) {
    return find_seq<false>(p, [&](int, int cu) { return cu <= t; }, index);
}

// Sequence i.
__device__ __forceinline__ Seq seq_at(const AttnParams &p, int i) {
    auto clamp = [](int x, int a, int b) { return min(max(x, a), b); };
    const int q_at = clamp(p.cu_q[i], 0, (int)p.total_q), k_at = clamp(p.cu_k[i], 0, (int)p.total_k);
    Seq s;
    s.q0 = q_at, s.k0 = k_at;
    s.lq = clamp(p.cu_q[i + 1], q_at, (int)p.total_q) - q_at;
    s.lk_slot = clamp(p.cu_k[i + 1], k_at, (int)p.total_k) - k_at;
    s.lk = p.len_k ? clamp(p.len_k[i], 0, s.lk_slot) : s.lk_slot;
    return s;
}

// packed row -> token (rows are below 2^31; most groups are powers of two)
__device__ __forceinline__ int row_token(const AttnParams &p, int row) {
    return p.lgrp >= 0 ? row >> p.lgrp : (int)((uint32_t)row / (uint32_t)p.grp);
}

// The packed rows of one wave (32 columns) of a row tile: this lane's row, and the keys its rows see.
struct Rows {
    bool live;
    int tok, hq;         // token in the sequence, query head (of a row past the end: the last one's)
    int last;            // last key this lane's row sees, -1: none
    int wave_min;        // the least `last` of the wave's live rows: tiles wholly up to it need no mask
    int wave_max;        // the largest, -1: the wave has no work
    int k_end;           // keys that some row of the workgroup sees
    int all;             // the last key that every row of the workgroup sees
};
__device__ __forceinline__ Rows rows_of(const AttnParams &p, const Seq &sq, int hk, int row_wg, int BM, int wave, int lane) {
    Rows r;
    const int end = sq.lq * p.grp, off = sq.lk - sq.lq;
    auto last_of = [&](int row) { return p.causal ? max(-1, min(row_token(p, row) + off, sq.lk - 1)) : sq.lk - 1; };
    const int first = row_wg + wave * 32, row = first + (lane & 31), at = min(row, end - 1);
    r.live = row < end;
    r.tok = row_token(p, at);
    r.hq = hk * p.grp + (at - r.tok * p.grp);
    r.last = !r.live ? -1 : p.causal ? max(-1, min(r.tok + off, sq.lk - 1)) : sq.lk - 1;
    // rows see longer and longer prefixes, so the wave's ends decide
    r.wave_min = first < end ? last_of(first) : -1;
    if (first + 32 > end) r.wave_min = -1;  // rows past the end see nothing
    r.wave_max = first < end ? last_of(min(first + 31, end - 1)) : -1;
    r.k_end = last_of(min(row_wg + BM, end) - 1) + 1;
    r.all = last_of(row_wg);
    return r;
}

// ---- which tile a workgroup takes ----
//
// Workgroups go round-robin over the 8 XCDs, each with an L2 of its own, and the tiles of one sequence and head
// read the same keys. Units are ordered (run of slots, head, slot of the run) and a run goes to one XCD: short
// sequences have their tiles in one run, one after the other; long ones (run = 1) go slot by slot over all heads, so
// that every head's longest causal tiles come first and, with a multiple of 8 heads, a head stays on its XCD.
constexpr int kXcds = 8;
__host__ __device__ __forceinline__ int64_t xcd_grid(int64_t slots, int heads, int run) {
    const int64_t units = (slots + run - 1) / run * run * heads, round = (int64_t)kXcds * run;
    return (units + round - 1) / round * round;
}
// (slot, head) of a workgroup; a slot past the last means none
__device__ __forceinline__ int64_t xcd_slot(uint32_t wg, int heads, int run, int &head) {
    const uint32_t x = wg & (kXcds - 1), pos = wg / kXcds, r = pos / (uint32_t)run, k = pos - r * (uint32_t)run;
    const uint32_t t = r * kXcds + x, g = t / (uint32_t)heads;
    head = (int)(t - g * (uint32_t)heads);
    return (int64_t)g * run + k;
}

}  // namespace eqlin

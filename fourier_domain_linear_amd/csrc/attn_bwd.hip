// attn_bwd.hip -- gradients of the packed attention. With P = exp(scale q k^T - lse) recomputed from the
// forward's lse, dP = dO V^T and delta = sum over d of dO O:
//
//   dS = P (dP - delta);  dV = P^T dO;  dK = scale dS^T Q;  dQ = scale dS K
//
// Two passes, each owning its outputs: one over row tiles (dQ, and delta for the other) and one over key tiles (dK,
// dV: every row that sees them, all heads of the group, in order). S and dP are formed in both, 7 products instead of
// 5, and nothing is added by atomics: the same bits every time, and no fp32 image of dQ in memory. P and dS are rounded to
// the half types as operands of their products, dS after the subtraction; all else is fp32.
//
// dQ is bound as the forward is; dK and dV at 128 dims by one wave's chain of reads, products and exponentials (below).
// 4 x 4096 tokens, 16 heads, bf16, every key seen: 2200 us at 128 dims (625 TFLOP/s of the formula's 5 products, 875 of the
// 7 formed; a large matrix product 1100), 965 us at 64 (712 and 997). Launches that do not fill the card split dq's keys and
// the rows of dk's and dv's key tiles, as partial sums in fp32 that k_attn_sum adds in order.
#include "attn.h"
#include "attn_tile.h"

namespace eqlin {

namespace {

// ---- fp16: where P and dS lie in the type's range ----
//
// Over thousands of keys P falls below fp16's normal range (2^-14), dS follows d_o down to nothing, and with a large loss
// scale it passes 65504. P enters its product times 2^8: with all its bits down to 2^-22, and in range where lse's rounding
// leaves it above 1 (scores in the millions). dS enters times a gain, a power of two of its own for each column (the query
// of dQ, the key of dK): it starts so high that the first block with a gradient lowers it, to a largest value of 2^8 to
// 2^9, and is lowered again, the sums so far with it, by a block that passes 2^15. Values down to 2^-23 of a column's
// largest so keep all their bits, and the stores divide by the gain. (bf16 has the range of fp32.) The price, 4 x 4096
// tokens, 16 heads, forward and gradients: 2907 us against 2866 us without it at 128 dims, 1456 against 1362 at 64.
template <class E>
constexpr bool kHasGain = __is_same(E, F16);
template <class E>
constexpr int kPGain = kHasGain<E> ? 8 : 0;  // (log2)
constexpr float kTop = 32768.0f;
constexpr int kAim = 9, kFirstGain = 60;  // (log2; the largest dS of fp16 operands is about 2^40)

__device__ __forceinline__ float abs_max(const f32x16 &x) {
    float m = 0.0f;
#pragma unroll
    for (int v = 0; v < 16; ++v) m = fmaxf(m, fabsf(x[v]));
    return m;
}
// The power of two that a column whose largest value is m is to be multiplied by.
__device__ __forceinline__ int lower_by(float m) { return m > kTop && m < INFINITY ? kAim - __builtin_amdgcn_frexp_expf(m) : 0; }

// ---- dQ: as the forward, 32 rows a wave (columns), key tiles through LDS ----
// (16 heads on 4 of 128 dims, bf16, 4 causal sequences up to 4096, 3000 on average: 289 us of the backward's 890)

// gain: log2 of the column's gain (0 but in fp16); lse2 is less it, so that the exponential brings it in.
template <class E, int DP, int NKB>
__device__ __forceinline__ void dq_block(f32x16 *dq, const uint4 *qf, const uint4 *gf, const typename Tile<E, DP>::Lane &L, uint32_t kt,
                                         uint32_t vt, float c, float &lse2, float &gain, float delta, bool masked, int lim, int h) {
    typedef Tile<E, DP> TL;
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb) {
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int t = 0; t < TL::kSteps; ++t) {
            s = mma_frag<E>(TL::row_frag(kt, L, kb, t), qf[t], s);
            dp = mma_frag<E>(TL::row_frag(vt, L, kb, t), gf[t], dp);
        }
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const float pr = __builtin_amdgcn_exp2f(fmaf(s[v], c, -lse2));
            s[v] = pr * (dp[v] - delta);
        }
        if (masked) {
#pragma unroll
            for (int v = 0; v < 16; ++v) s[v] = 32 * kb + d_row(v, 0) <= lim - 4 * h ? s[v] : 0.0f;
        }
        if constexpr (kHasGain<E>) {
            const float m = abs_max(s);
            if (__any(m > kTop)) {
                const int by = lower_by(half_max(m));
                const float r = ldexpf(1.0f, by);
                gain += by, lse2 -= by;
#pragma unroll
                for (int v = 0; v < 16; ++v) s[v] *= r;
#pragma unroll
                for (int db = 0; db < DP / 32; ++db)
#pragma unroll
                    for (int v = 0; v < 16; ++v) dq[db][v] *= r;
            }
        }
        WFrags<E> w;
        w.set(s);
#pragma unroll
        for (int f = 0; f < WFrags<E>::NF; ++f)
#pragma unroll
            for (int db = 0; db < DP / 32; ++db)
                dq[db] = mma_frag<E>(TL::col_frag(kt, L, kb, f, db), w.f[f], dq[db]);
    }
}

// delta of rows that see no key past the first tile: sum over its keys of P dP, in fp32 throughout. Over a handful of
// keys (short sequences, a causal sequence's first rows) the sum of dO O carries o's rounding into the gradients about
// as far as their own rounding; over more it is lost among the terms (unless the values share a part many times their spread:
// it is u |o| |dO|, they are as dP - delta). A row that sees one key has P = 1 and so dS = 0,
// exactly.
template <class E, int DP, int NKB>
__device__ __forceinline__ float delta_of_tile(const uint4 *qf, const uint4 *gf, const typename Tile<E, DP>::Lane &L, uint32_t kt,
                                               uint32_t vt, float c, float lse2, int lim, int h) {
    typedef Tile<E, DP> TL;
    float sum = 0.0f;
#pragma unroll 1
    for (int kb = 0; kb < NKB; ++kb) {
        const uint32_t at = kb * 32 * TL::kRow;
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int t = 0; t < TL::kSteps; ++t) {
            s = mma_frag<E>(TL::row_frag(kt + at, L, 0, t), qf[t], s);
            dp = mma_frag<E>(TL::row_frag(vt + at, L, 0, t), gf[t], dp);
        }
#pragma unroll
        for (int v = 0; v < 16; ++v)
            sum += 32 * kb + d_row(v, 0) <= lim - 4 * h ? (lim == 0 ? 1.0f : __builtin_amdgcn_exp2f(fmaf(s[v], c, -lse2))) * dp[v] : 0.0f;
    }
    return half_sum(sum);
}

// Partial sums in fp32 (shares of dq, or of dk and then dv) lie behind delta in the workspace.
__host__ __device__ __forceinline__ int64_t share_offset(const AttnParams &p) { return (p.total_q * p.Hq + 63) / 64 * 64; }

// SPLIT: a workgroup takes one of p.nsplit ranges of its keys; range 0 has the first tile wherever there is one, and so the
// delta of rows that see few keys. (Its own instance: the range's registers cost the launches that fill the card without it
// 8 % at 128 dims.)
template <class E, int DP, bool SPLIT>
__global__ void __launch_bounds__(256, __is_same(E, F32) ? 1 : 2) k_attn_dq(const AttnParams p) {
    typedef TileCfg<E, DP> C;
    typedef Tile<E, DP> TL;
    typedef typename ElemOf<E>::type T;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;
    int hk;
    const int64_t slot = p.slots - 1 - xcd_slot(blockIdx.x, p.Hkv, p.run, hk);  // causal: a sequence's longest rows first
    if (slot < 0) return;
    int64_t tile;
    const Seq sq = seq_of_slot<false>(p, p.grp, C::BM, slot, tile);
    const int row_wg = (int)tile * C::BM;
    if (tile < 0 || row_wg >= sq.lq * p.grp) return;
    const Rows r = rows_of(p, sq, hk, row_wg, C::BM, wave, lane);
    int beg = 0, end = r.k_end;
    if constexpr (SPLIT) {
        const int tiles = (end + C::BN - 1) / C::BN, z = blockIdx.z;
        auto first_of = [&](int i) { return (int)(((int64_t)tiles * i + p.nsplit - 1) / p.nsplit) * C::BN; };
        beg = first_of(z);
        end = min(end, first_of(z + 1));
    }
    const int k_beg = SPLIT ? beg : 0, k_end = SPLIT ? end : r.k_end;
    const T *kg = (const T *)p.k + sq.k0 * p.kt + hk * p.kh;
    const T *vg = (const T *)p.v + sq.k0 * p.vt + hk * p.vh;
    TileDma<E, DP, C::BN> tk, tv;
    const uint32_t lds0 = lds_offset(lds);
    auto fetch = [&](int k0, int buf) {
        const int valid = sq.lk - k0;
        if (valid < C::BN) {
            tk.offsets(p.kt, valid, wave, lane);
            tv.offsets(p.vt, valid, wave, lane);
        }
        tk.issue(lds0 + buf * 2 * C::kTileBytes, kg + (int64_t)k0 * p.kt, p.D, wave, lane);
        tv.issue(lds0 + buf * 2 * C::kTileBytes + C::kTileBytes, vg + (int64_t)k0 * p.vt, p.D, wave, lane);
    };
    zero_pad(lds, C::kLds, p.D, DP, tid);
    tk.offsets(p.kt, C::BN, wave, lane);
    tv.offsets(p.vt, C::BN, wave, lane);
    if (k_beg < k_end) fetch(k_beg, 0);
    const int64_t at = (sq.q0 + r.tok) * p.Hq + r.hq;
    uint4 qf[TL::kSteps], gf[TL::kSteps];
    load_row<E, DP>(qf, (const T *)p.q + (sq.q0 + r.tok) * p.qt + r.hq * p.qh, p.D, h);
    load_row<E, DP>(gf, (const T *)p.dout + (sq.q0 + r.tok) * p.dot + r.hq * p.doh, p.D, h);
    float lse2 = p.lse[at] * kLog2e, gain = kHasGain<E> ? kFirstGain : 0;
    // delta = sum over d of dO O, here and for the other pass
    float delta = 0.0f;
    {
        uint4 of[TL::kSteps];
        load_row<E, DP>(of, (const T *)p.o + (sq.q0 + r.tok) * p.ot + r.hq * p.oh, p.D, h);
#pragma unroll
        for (int t = 0; t < TL::kSteps; ++t) {
            float a[Elem<E>::V], b[Elem<E>::V];
            Elem<E>::unpack(of[t], a);
            Elem<E>::unpack(gf[t], b);
#pragma unroll
            for (int j = 0; j < Elem<E>::V; ++j) delta = fmaf(a[j], b[j], delta);
        }
        delta = half_sum(delta);
    }
    f32x16 dq[DP / 32];
#pragma unroll
    for (int db = 0; db < DP / 32; ++db) dq[db] = zero16();
    const float c = p.scale * kLog2e;
    const typename TL::Lane L = TL::lane_of(lane);
    int buf = 0;
    int *flags = (int *)(lds + C::kLds);
    bool bad = false;  // some tile was cleared
    auto arrive = [&](int k0) {
        dma_wait();
        __syncthreads();  // this tile is in LDS; the other buffer has no more readers
        if (k0 + C::BN < k_end) fetch(k0 + C::BN, buf ^ 1);
        if (k0 + C::BN - 1 > r.all) {  // some row sees only part of it (uniform in the workgroup)
            char *kt = lds + 2 * buf * C::kTileBytes;
            const bool mine = __any(tile_nonfinite<E, 256>(kt, C::kTileBytes, tid));
            if (lane == 0) flags[4 * buf + wave] = mine;
            __syncthreads();
            if (uniform(flags[4 * buf] | flags[4 * buf + 1] | flags[4 * buf + 2] | flags[4 * buf + 3])) {
                bad = true;
                clear_nonfinite<E, 256>(kt, C::kTileBytes, tid);
                __syncthreads();
            }
        }
    };
    if (k_beg < k_end && r.wave_max >= k_beg) {
        arrive(k_beg);
        if (k_beg == 0 && uniform(r.last) < C::BN) {  // the wave's first row, which sees least
            const float d = delta_of_tile<E, DP, C::NKB>(qf, gf, L, lds0, lds0 + C::kTileBytes, c, lse2, r.last, h);
            delta = r.last < C::BN ? d : delta;
        }
        lse2 -= gain;
        for (int k0 = k_beg;;) {
            const uint32_t kt = lds0 + buf * 2 * C::kTileBytes, vt = kt + C::kTileBytes;
            dq_block<E, DP, C::NKB>(dq, qf, gf, L, kt, vt, c, lse2, gain, delta, k0 + C::BN - 1 > r.wave_min, r.last - k0, h);
            buf ^= 1;
            if ((k0 += C::BN) >= k_end) break;
            arrive(k0);
        }
    } else {  // a wave without rows or keys fetches its part of the tiles
        for (int k0 = k_beg; k0 < k_end; k0 += C::BN) {
            arrive(k0);
            buf ^= 1;
        }
    }
    if (r.live && h == 0 && (!SPLIT || blockIdx.z == 0)) p.ws[at] = delta;
    if (bad)
        poison_columns<E, DP>(dq, k_beg + max(0, r.all + 1 - k_beg) / C::BN * C::BN, min(r.wave_max, k_end - 1), p.D, h,
                              [&](int j) { return kg + (int64_t)j * p.kt; }, [&](int j) { return j <= r.last; });
    if (!r.live) return;
    const float scale = kHasGain<E> ? ldexpf(p.scale, -(int)gain) : p.scale;
    if constexpr (SPLIT)  // fp32, for k_attn_sum
        store_column<F32, DP>(dq, scale, p.ws + share_offset(p) + (blockIdx.z * p.total_q * p.Hq + at) * p.D, p.D, h);
    else
        store_column<E, DP>(dq, scale, (T *)p.dq + (sq.q0 + r.tok) * p.dqt + r.hq * p.dqh, p.D, h);
}

// ---- dK, dV: 32 keys a wave (columns), tiles of packed rows (q and dO) through LDS ----
//
// The keys' operands and dk and dv stay in a wave's registers: at 128 dims 192 of the 383 in use, one wave a SIMD, whose
// exponentials wait for its products and its products for its reads: matrix cores 29 % busy, LDS 19 %, no bank conflicts.
// (Two waves a SIMD, with the keys in LDS, read half as much again and take the same time: 2171 us for the backward
// above, against 2196 us.) The sequences above: 550 us of 890, and 45 us for the sum of the shares.

// One group of the products that reduce over the tile's rows: the DP / 32 A fragments of reduction step f.
template <class E, int DP>
struct ColGroup {
    uint4 a[DP / 32];
    __device__ __forceinline__ void load(uint32_t tile, const typename Tile<E, DP>::Lane &L, int blk, int f) {
#pragma unroll
        for (int db = 0; db < DP / 32; ++db) a[db] = Tile<E, DP>::col_frag(tile, L, blk, f, db);
    }
    __device__ __forceinline__ void multiply(f32x16 *acc, const uint4 &w) const {
#pragma unroll
        for (int db = 0; db < DP / 32; ++db) acc[db] = mma_frag<E>(a[db], w, acc[db]);
    }
};

template <class E, int DP, int NRB>
__device__ __forceinline__ void dkv_block(f32x16 *dk, f32x16 *dv, const uint4 *kf, const uint4 *vf,
                                          const typename Tile<E, DP>::Lane &L, uint32_t qt, uint32_t gt, uint32_t stats, float c,
                                          float &gain, bool masked, int key, int h) {
    typedef Tile<E, DP> TL;
    constexpr int BR = 32 * NRB, NF = WFrags<E>::NF;
#pragma unroll
    for (int rb = 0; rb < NRB; ++rb) {
        const uint32_t at = stats + 16 * h + 32 * rb * 4;
        f32x16 s = zero16(), dp = zero16();
        f32x4 ls[4], de[4];
        uint4 qa[TL::kSteps], ga[TL::kSteps];
#pragma unroll
        for (int t = 0; t < TL::kSteps; ++t) {
            qa[t] = TL::row_frag(qt, L, rb, t);
            ga[t] = TL::row_frag(gt, L, rb, t);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            ls[g] = TL::template lds_at<f32x4>(at + 32 * g);
            de[g] = TL::template lds_at<f32x4>(at + 32 * g + BR * 4);
        }
#pragma unroll
        for (int t = 0; t < TL::kSteps; ++t) {
            s = mma_frag<E>(qa[t], kf[t], s);
            dp = mma_frag<E>(ga[t], vf[t], dp);
        }
        ColGroup<E, DP> g0, g1;
        g0.load(gt, L, rb, 0);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = 4 * g + j;
                s[v] = __builtin_amdgcn_exp2f(fmaf(s[v], c, -ls[g][j]));
                dp[v] = s[v] * (dp[v] - de[g][j]);
            }
        }
        if (masked) {
            typedef int i32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const i32x4 la = TL::template lds_at<i32x4>(at + 32 * g + 2 * BR * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int v = 4 * g + j;
                    s[v] = key <= la[j] ? s[v] : 0.0f;
                    dp[v] = key <= la[j] ? dp[v] : 0.0f;
                }
            }
        }
        if constexpr (kHasGain<E>) {
            const float m = abs_max(dp) * gain;
            if (__any(m > kTop)) {
                const float r = ldexpf(1.0f, lower_by(half_max(m)));
                gain *= r;
#pragma unroll
                for (int db = 0; db < DP / 32; ++db)
#pragma unroll
                    for (int v = 0; v < 16; ++v) dk[db][v] *= r;
            }
#pragma unroll
            for (int v = 0; v < 16; ++v) dp[v] *= gain;
        }
        WFrags<E> w, w2;
        w.set(s);
        w2.set(dp);
#pragma unroll
        for (int i = 0; i < 2 * NF; ++i) {  // dv over dO's fragments, then dk over q's
            if (i + 1 < 2 * NF) g1.load(i + 1 < NF ? gt : qt, L, rb, (i + 1) % NF);
            if (i < NF) g0.multiply(dv, w.f[i]);
            else g0.multiply(dk, w2.f[i - NF]);
            g0 = g1;
        }
    }
}

template <class E, int DP>
struct DkvCfg {
    typedef Tile<E, DP> TL;
    static constexpr int BK = 128;  // keys of a workgroup
    static constexpr int NRB = __is_same(E, F32) ? 1 : 2;
    static constexpr int BR = 32 * NRB;  // packed rows of a tile
    static constexpr int kTileBytes = BR * TL::kRow;
    static constexpr int kStats = 3 * BR * 4;                    // lse, delta, last key of each row
    static constexpr int kFlags = 4 * 4;                         // a word a wave
    static constexpr int kLds = 4 * kTileBytes + 2 * (kStats + kFlags);  // q and dO, two buffers; then the rows' values
};

template <class E, int DP>
__global__ void __launch_bounds__(256, __is_same(E, F32) || DP > 64 ? 1 : 2) k_attn_dkv(const AttnParams p) {
    typedef DkvCfg<E, DP> C;
    typedef Tile<E, DP> TL;
    typedef typename ElemOf<E>::type T;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;
    int hz;
    const int64_t slot = xcd_slot(blockIdx.x, p.Hkv * p.nsplit, p.run, hz);  // causal: a sequence's first keys have most rows
    const int hk = hz % p.Hkv, z = hz / p.Hkv;
    if (slot >= p.slots) return;
    int64_t tile;
    const Seq sq = seq_of_slot<true>(p, 1, C::BK, slot, tile);
    const int64_t key_wg = tile * C::BK;
    if (key_wg < 0 || key_wg >= sq.lk_slot) return;
    const int off = sq.lk - sq.lq;
    const int key = (int)key_wg + wave * 32 + (lane & 31);
    const int key_at = min(key, sq.lk_slot - 1);
    uint4 kf[TL::kSteps], vf[TL::kSteps];
    load_row<E, DP>(kf, (const T *)p.k + (sq.k0 + key_at) * p.kt + hk * p.kh, p.D, h);
    load_row<E, DP>(vf, (const T *)p.v + (sq.k0 + key_at) * p.vt + hk * p.vh, p.D, h);
    f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int db = 0; db < DP / 32; ++db) dk[db] = zero16(), dv[db] = zero16();
    const float c = p.scale * kLog2e;
    const int64_t rows = key_wg < sq.lk ? (int64_t)sq.lq * p.grp : 0;
    // causal: the first token that sees the workgroup's first key
    int64_t row_beg = p.causal && key_wg > off ? (key_wg - off) * p.grp : 0;
    row_beg -= row_beg % C::BR;
    // this workgroup's share of the rows, in whole tiles
    int64_t row_end = rows;
    if (p.nsplit > 1 && row_beg < rows) {
        const int64_t tiles = (rows - row_beg + C::BR - 1) / C::BR;
        row_end = min(rows, row_beg + tiles * (z + 1) / p.nsplit * C::BR);
        row_beg += tiles * z / p.nsplit * C::BR;
    }
    const T *qg = (const T *)p.q + sq.q0 * p.qt + (int64_t)hk * p.grp * p.qh;
    const T *gg = (const T *)p.dout + sq.q0 * p.dot + (int64_t)hk * p.grp * p.doh;
    const float *lse = p.lse + sq.q0 * p.Hq + hk * p.grp, *del = p.ws + sq.q0 * p.Hq + hk * p.grp;
    TileDma<E, DP, C::BR> tq, tg;
    const uint32_t lds0 = lds_offset(lds);
    const typename TL::Lane L = TL::lane_of(lane);
    float st_lse = INFINITY, st_del = 0.0f, gain = kHasGain<E> ? ldexpf(1.0f, kFirstGain - kPGain<E>) : 1.0f;
    int st_last = -1;
    // Row offsets within a tile repeat from tile to tile where the group divides the tile.
    const bool repeats = C::BR % p.grp == 0;
    auto load = [&](int64_t r0, int buf) {
        const int tok0 = (int)((uint32_t)r0 / (uint32_t)p.grp), rem = (int)((uint32_t)r0 - (uint32_t)tok0 * (uint32_t)p.grp);
        const int64_t valid = row_end - r0;
        if (!repeats || valid < C::BR) {
            tq.offsets_packed(p.qt, p.qh, rem, p.grp, (int)min(valid, (int64_t)C::BR), wave, lane);
            tg.offsets_packed(p.dot, p.doh, rem, p.grp, (int)min(valid, (int64_t)C::BR), wave, lane);
        }
        tq.issue(lds0 + 2 * buf * C::kTileBytes, qg + tok0 * p.qt, p.D, wave, lane);
        tg.issue(lds0 + (2 * buf + 1) * C::kTileBytes, gg + tok0 * p.dot, p.D, wave, lane);
        if (tid < C::BR) {
            const uint32_t r = (uint32_t)(rem + tid);
            const int tok = tok0 + (int)(r / (uint32_t)p.grp), hh = (int)(r % (uint32_t)p.grp);
            const bool in = tid < valid;
            st_lse = in ? lse[(int64_t)tok * p.Hq + hh] * kLog2e - kPGain<E> : INFINITY;
            st_del = in ? del[(int64_t)tok * p.Hq + hh] : 0.0f;
            st_last = in ? (p.causal ? min(tok + off, sq.lk - 1) : sq.lk - 1) : -1;
        }
    };
    auto store = [&](int buf) {
        if (tid < C::BR) {
            float *f = (float *)(lds + 4 * C::kTileBytes + buf * (C::kStats + C::kFlags));
            f[tid] = st_lse;
            f[C::BR + tid] = st_del;
            ((int *)f)[2 * C::BR + tid] = st_last;
        }
    };
    zero_pad(lds, C::kLds, p.D, DP, tid);
    if (row_beg < row_end) {
        tq.offsets_packed(p.qt, p.qh, 0, p.grp, C::BR, wave, lane);
        tg.offsets_packed(p.dot, p.doh, 0, p.grp, C::BR, wave, lane);
        load(row_beg, 0);
        store(0);
    }
    int buf = 0;
    const int wave_last = (int)key_wg + wave * 32 + 31;  // the wave's last key
    const int wg_last = min((int)key_wg + C::BK, sq.lk) - 1;  // the workgroup's last key that counts
    int bad_from = -1, bad_to = -1;  // rows of tiles that were cleared
    for (int64_t r0 = row_beg; r0 < row_end; r0 += C::BR) {
        dma_wait();
        __syncthreads();
        const bool more = r0 + C::BR < row_end;
        if (more) load(r0 + C::BR, buf ^ 1);
        const uint32_t qt = lds0 + 2 * buf * C::kTileBytes, gt = qt + C::kTileBytes, stats = lds0 + 4 * C::kTileBytes + buf * (C::kStats + C::kFlags);
        // rows see a prefix of the keys, longer for later rows: the tile's first row decides
        const int first_sees = uniform(TL::template lds_at<int>(stats + 2 * C::BR * 4));
        const bool whole = first_sees >= wave_last && r0 + C::BR <= row_end;
        if (first_sees < wg_last || r0 + C::BR > row_end) {  // some key is not seen by all its rows (uniform in the workgroup)
            int *flags = (int *)(lds + 4 * C::kTileBytes + buf * (C::kStats + C::kFlags) + C::kStats);
            char *tile = lds + 2 * buf * C::kTileBytes;
            const bool mine = __any(tile_nonfinite<E, 256>(tile, 2 * C::kTileBytes, tid));
            if (lane == 0) flags[wave] = mine;
            __syncthreads();
            if (uniform(flags[0] | flags[1] | flags[2] | flags[3])) {
                if (bad_from < 0) bad_from = (int)r0;
                bad_to = (int)min(r0 + C::BR, row_end) - 1;
                clear_nonfinite<E, 256>(tile, 2 * C::kTileBytes, tid);
                __syncthreads();
            }
        }
        dkv_block<E, DP, C::NRB>(dk, dv, kf, vf, L, qt, gt, stats, c, gain, !whole, key, h);
        if (more) store(buf ^ 1);
        buf ^= 1;
    }
    if (bad_from >= 0)  // (q's values that are not finite reach dk and dv through lse, dO's reach dk through delta)
        add_nonfinite<E, DP>(dv, bad_from, bad_to, p.D, h,
                             [&](int row) {
                                 const int t = row_token(p, row);
                                 return gg + (int64_t)t * p.dot + (row - t * p.grp) * p.doh;
                             },
                             [&](int row) { return !p.causal || key <= row_token(p, row) + off; });
    if (key >= sq.lk_slot) return;
    if (key >= sq.lk) {  // beyond the sequence's length in its slot: zeros
#pragma unroll
        for (int db = 0; db < DP / 32; ++db) dk[db] = zero16(), dv[db] = zero16();
    }
    const float dk_scale = kHasGain<E> ? ldexpf(p.scale, -kPGain<E>) / gain : p.scale, dv_scale = ldexpf(1.0f, -kPGain<E>);
    if (p.nsplit > 1) {  // a share: fp32, for k_attn_sum
        const int64_t heads = p.total_k * p.Hkv, at = (sq.k0 + key) * p.Hkv + hk;
        float *part = p.ws + share_offset(p);
        store_column<F32, DP>(dk, dk_scale, part + (z * heads + at) * p.D, p.D, h);
        store_column<F32, DP>(dv, dv_scale, part + ((p.nsplit + z) * heads + at) * p.D, p.D, h);
        return;
    }
    store_column<E, DP>(dk, dk_scale, (T *)p.dk + (sq.k0 + key) * p.dkt + hk * p.dkh, p.D, h);
    store_column<E, DP>(dv, dv_scale, (T *)p.dv + (sq.k0 + key) * p.dvt + hk * p.dvh, p.D, h);
}

// out[token][head][.] = sum of the n partial results, in order: four values a thread. The parts of a second tensor lie
// behind those of the first. Sequences are stretches one behind the other, so a token in front of the first bound or from
// the last on is none's: nobody wrote its parts, and it is left as it is.
struct Sum {
    const float *part;
    const int *cu;
    int B;
    int64_t heads;  // tokens * H
    int n, H, D;
    void *out[2];
    int64_t ts[2], hs[2];
};
template <class E>
__global__ void __launch_bounds__(256) k_attn_sum(const Sum p) {
    typedef typename ElemOf<E>::type T;
    const int per = p.D / 4, w = blockIdx.y, begin = p.cu[0], end = p.cu[p.B];
    const int64_t n = p.heads * per, part = p.heads * p.D;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t at = i / per, t = at / p.H;
        if (t < begin || t >= end) continue;
        const int d = (int)(i - at * per) * 4;
        const float *src = p.part + w * p.n * part + at * p.D + d;
        float4 s = *(const float4 *)src;
        for (int z = 1; z < p.n; ++z) {
            const float4 a = *(const float4 *)(src + z * part);
            s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
        }
        T *dst = (T *)p.out[w] + t * p.ts[w] + (at - t * p.H) * p.hs[w] + d;
        if constexpr (__is_same(E, F32)) *(float4 *)dst = s;
        else *(uint2 *)dst = make_uint2(pack2<E>(s.x, s.y), pack2<E>(s.z, s.w));
    }
}
template <class E>
void run_sum(const Sum &p, int tensors, hipStream_t s) {
    const int64_t n = p.heads * (p.D / 4);
    hipLaunchKernelGGL((k_attn_sum<E>), dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 16), tensors), dim3(256), 0, s, p);
}

// Key ranges that dq's row tiles are split into, where those do not fill the card: none shorter than 256 keys on average
// (fp32, whose products take eight times as long: 64). One sequence of 1454, 2 heads on 1 of 40 dims, fp16: the backward in
// 36 us, against 56 us unsplit; of 2827, 3 heads of 128, fp32: 461 us, against 809 us.
int pick_ranges(const AttnParams &p, bool half) {
    const int64_t wgs = std::max<int64_t>(1, (p.total_q * p.grp / 128 + p.B) * p.Hkv), want = 2 * (int64_t)device_num_cus();
    const int64_t most = p.total_k / std::max(1, p.B) / (half ? 256 : 64);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want / wgs, most), 8));
}

// Shares that the rows of a key tile are split into, where the key tiles alone do not fill the card: a tile of a
// causal sequence's first keys with grouped heads has thousands of rows, and one workgroup with them all is the
// launch's whole time (4 sequences up to 4096, 16 heads on 4: 975 us in one share, 947 in 3, 888 in 6; shares of one
// length instead, fewer for a tile of fewer rows, leave a longer tail: 900 to 920 us). Up to two workgroups a compute unit
// shares go down to 64 rows (4 sequences up to 597, 8 heads on 2 of 64: 40 us, against 82 us in one).
int pick_shares(const AttnParams &p) {
    const int64_t wgs = std::max<int64_t>(1, (p.total_k / 128 + p.B) * p.Hkv), cus = device_num_cus();
    const int64_t rows = p.total_q * p.grp / std::max(1, p.B);  // of a sequence on average
    const int64_t n = std::max(std::min(8 * cus / wgs, rows / 512), std::min(2 * cus / wgs, rows / 64));
    return (int)std::max<int64_t>(1, std::min<int64_t>(n, 8));
}

template <class K>
hipError_t set_lds(K kernel, int bytes) {
    return bytes > 64 * 1024 ? hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes)
                             : hipSuccess;
}

template <class E, int DP>
hipError_t run_bwd(const AttnParams &p0, hipStream_t s) {
    AttnParams p = p0;
    typedef TileCfg<E, DP> CQ;
    typedef DkvCfg<E, DP> CK;
    hipError_t e = set_lds(k_attn_dq<E, DP, false>, CQ::kLds + CQ::kFlags);
    if (e == hipSuccess) e = set_lds(k_attn_dq<E, DP, true>, CQ::kLds + CQ::kFlags);
    if (e == hipSuccess) e = set_lds(k_attn_dkv<E, DP>, CK::kLds);
    if (e != hipSuccess) return e;
    if (p.total_q > 0) {
        p.slots = p.total_q * p.grp / CQ::BM + p.B;
        p.run = run_of(p.slots, p.B);
        p.nsplit = pick_ranges(p, !__is_same(E, F32));
        const dim3 grid((unsigned)xcd_grid(p.slots, p.Hkv, p.run), 1, p.nsplit);
        if (p.nsplit > 1) {
            hipLaunchKernelGGL((k_attn_dq<E, DP, true>), grid, dim3(256), CQ::kLds + CQ::kFlags, s, p);
            run_sum<E>({p.ws + share_offset(p), p.cu_q, p.B, p.total_q * p.Hq, p.nsplit, p.Hq, p.D, {p.dq}, {p.dqt}, {p.dqh}}, 1, s);
        } else {
            hipLaunchKernelGGL((k_attn_dq<E, DP, false>), grid, dim3(256), CQ::kLds + CQ::kFlags, s, p);
        }
    }
    if (p.total_k > 0) {
        p.slots = p.total_k / CK::BK + p.B;
        p.run = run_of(p.slots, p.B);
        p.nsplit = pick_shares(p);
        hipLaunchKernelGGL((k_attn_dkv<E, DP>), dim3((unsigned)xcd_grid(p.slots, p.Hkv * p.nsplit, p.run)), dim3(256), CK::kLds, s, p);
        if (p.nsplit > 1)
            run_sum<E>({p.ws + share_offset(p), p.cu_k, p.B, p.total_k * p.Hkv, p.nsplit, p.Hkv, p.D, {p.dk, p.dv}, {p.dkt, p.dvt}, {p.dkh, p.dvh}}, 2, s);
    }
    return hipGetLastError();
}

template <class E>
hipError_t run_bwd_e(const AttnParams &p, hipStream_t s) {
    if (p.D <= 32) return run_bwd<E, 32>(p, s);
    if (p.D <= 64) return run_bwd<E, 64>(p, s);
    return run_bwd<E, 128>(p, s);
}

}  // namespace

size_t attention_backward_workspace_bytes(const AttnParams &p, eqlin_dtype_t dtype) {
    if (p.B <= 0) return 0;
    const size_t n = pick_shares(p), shares = n > 1 ? 2 * n * p.total_k * p.Hkv * p.D : 0;
    const size_t m = pick_ranges(p, dtype != EQLIN_F32), ranges = m > 1 ? m * p.total_q * p.Hq * p.D : 0;
    return ((size_t)share_offset(p) + std::max(shares, ranges)) * sizeof(float);
}

hipError_t launch_attention_backward(const AttnParams &p, eqlin_dtype_t dtype, hipStream_t s) {
    if (dtype == EQLIN_F32) return run_bwd_e<F32>(p, s);
    if (dtype == EQLIN_F16) return run_bwd_e<F16>(p, s);
    return run_bwd_e<BF16>(p, s);
}

}  // namespace eqlin

// attn_fwd.hip -- attention over packed sequences: o = softmax(scale q k^T) v, one pass over the keys with
// the running maximum and sum.
//
// Bound by the matrix cores at 128 dims, and by the vector work beside them below: a 32 x 32 block of scores costs
// 16 products of 32 clocks at 128 dims and 8 at 64, and at both 16 exponentials of 16 clocks and about 100 other vector
// instructions of 4. 4 x 4096 tokens, 16 heads, bf16, every key seen: 520 to 600 us at 128 dims (0.92 to 1.05 PFLOP/s, by the
// card's clock; a large matrix product reaches 1.1), 306 to 335 us at 64 (0.82 to 0.90), 248 us at 32 (0.55). Sequences of
// different lengths are started in their packing's order, backwards: 24 of 403 to 3136, 6 heads of 64, 157 us with the
// longest packed last, 192 us with it first. fp32, 4096 tokens, 8 heads of 128: 607 us, 113 TFLOP/s (a matrix product: 153),
// matrix cores 68 % busy at one workgroup a compute unit.
#include "attn.h"
#include "attn_fwd.h"

namespace eqlin {

namespace {

// ---- the tile kernel: 4 waves, each 32 packed rows (the columns of S^T), all over the same key tiles ----
//
// A wave's rows stay in registers as operands, its results as accumulators; k and v tiles pass through two LDS buffers,
// the next one on its way while this one is multiplied. Four waves share a tile, so that its LDS reads (a fragment is
// read once a wave) stay below the products' time, and short sequences do not lose a larger tile's padding.

// Two shapes at DP = 128 in the half types. 64-key tiles at two waves a SIMD read V's fragments ahead of the
// exponentials and pay the running maximum once for 64 keys (4 x 4096 tokens, 16 heads: 562 us, against 581 for the
// other). Over few keys the launch is bound by each workgroup's chain of loads instead, and 32-key tiles, whose 16
// score registers less let three waves share a SIMD, are faster (64 x 196 tokens, 16 heads: 62 us against 71).
template <class E, int DP, bool SHORT>
struct FwdCfg {
    typedef Tile<E, DP> TL;
    static constexpr bool kSmall = SHORT && DP == 128;
    static constexpr int BM = 128;                                              // packed rows of a workgroup
    static constexpr int NKB = __is_same(E, F32) || kSmall ? 1 : 2;             // 32-key blocks of a tile
    static constexpr int BN = 32 * NKB;
    static constexpr int WPE = __is_same(E, F32) ? 1 : DP < 128 ? 4 : kSmall ? 3 : 2;          // waves a SIMD the registers allow
    static constexpr int kTileBytes = BN * TL::kRow;
    static constexpr int kLds = 4 * kTileBytes;                                 // k and v, two buffers;
    static constexpr int kFlags = 2 * 4 * 4;                                    // a word a wave, two sets
};
constexpr int64_t kShortKeys = 512;  // keys a sequence on average up to which SHORT is taken

template <class E, int DP, bool SHORT>
__global__ void __launch_bounds__(256, (FwdCfg<E, DP, SHORT>::WPE)) k_attn_fwd(const AttnParams p) {
    typedef FwdCfg<E, DP, SHORT> C;
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
    if (tile < 0 || row_wg >= sq.lq * p.grp || sq.lq * p.grp <= p.rcap) return;  // (so few rows: the step kernel's)
    const Rows r = rows_of(p, sq, hk, row_wg, C::BM, wave, lane);
    int k_beg = 0, k_end = r.k_end;
    if (p.nsplit > 1) {
        const int tiles = (k_end + C::BN - 1) / C::BN, z = blockIdx.z;
        k_beg = (int)((int64_t)tiles * z / p.nsplit) * C::BN;
        k_end = min(k_end, (int)((int64_t)tiles * (z + 1) / p.nsplit) * C::BN);
    }

    // the first tile's loads go first
    const T *kg = (const T *)p.k + sq.k0 * p.kt + hk * p.kh;
    const T *vg = (const T *)p.v + sq.k0 * p.vt + hk * p.vh;
    TileDma<E, DP, C::BN> dk, dv;
    const uint32_t lds0 = lds_offset(lds);
    auto fetch = [&](int k0, int buf) {
        const int valid = sq.lk - k0;
        if (valid < C::BN) {
            dk.offsets(p.kt, valid, wave, lane);
            dv.offsets(p.vt, valid, wave, lane);
        }
        dk.issue(lds0 + buf * 2 * C::kTileBytes, kg + (int64_t)k0 * p.kt, p.D, wave, lane);
        dv.issue(lds0 + buf * 2 * C::kTileBytes + C::kTileBytes, vg + (int64_t)k0 * p.vt, p.D, wave, lane);
    };
    zero_pad(lds, C::kLds, p.D, DP, tid);
    dk.offsets(p.kt, C::BN, wave, lane);
    dv.offsets(p.vt, C::BN, wave, lane);
    if (k_beg < k_end) fetch(k_beg, 0);
    uint4 qf[TL::kSteps];
    load_row<E, DP>(qf, (const T *)p.q + (sq.q0 + r.tok) * p.qt + r.hq * p.qh, p.D, h);

    FwdState<E, DP> st;
    st.clear();
    const float c = p.scale * kLog2e;

    const typename TL::Lane L = TL::lane_of(lane);
    int buf = 0;
    // (a wave without rows or keys fetches its part of the tiles, in a loop of its own)
    const bool works = r.wave_max >= k_beg;
    int *flags = (int *)(lds + C::kLds);
    bool bad = false;  // some tile was cleared
    auto arrive = [&](int k0) {
        dma_wait();
        __syncthreads();  // this tile is in LDS; the other buffer has no more readers
        if (k0 + C::BN < k_end) fetch(k0 + C::BN, buf ^ 1);
        if (k0 + C::BN - 1 > r.all) {  // some row sees only part of it (uniform in the workgroup)
            char *vt = lds + (2 * buf + 1) * C::kTileBytes;
            const bool mine = __any(tile_nonfinite<E, 256>(vt, C::kTileBytes, tid));
            if (lane == 0) flags[4 * buf + wave] = mine;
            __syncthreads();
            if (uniform(flags[4 * buf] | flags[4 * buf + 1] | flags[4 * buf + 2] | flags[4 * buf + 3])) {
                bad = true;
                clear_nonfinite<E, 256>(vt, C::kTileBytes, tid);
                __syncthreads();
            }
        }
    };
    if (works) {
        for (int k0 = k_beg; k0 < k_end; k0 += C::BN) {
            arrive(k0);
            const uint32_t kt = lds0 + buf * 2 * C::kTileBytes, vt = kt + C::kTileBytes;
            fwd_block<E, DP, C::NKB>(st, qf, L, kt, vt, c, k0 + C::BN - 1 > r.wave_min, r.last - k0, h);
            buf ^= 1;
        }
    } else {
        for (int k0 = k_beg; k0 < k_end; k0 += C::BN) {
            arrive(k0);
            buf ^= 1;
        }
    }

    if (bad)  // tiles begin at k_beg + BN i, and they were looked over from the one that holds key r.all + 1 on
        add_nonfinite<E, DP>(st.o, k_beg + max(0, r.all + 1 - k_beg) / C::BN * C::BN, min(r.wave_max, k_end - 1), p.D, h,
                             [&](int j) { return vg + (int64_t)j * p.vt; }, [&](int j) { return j <= r.last; });
    if (p.nsplit > 1) {  // partial results: unnormalised o, then (m, l), for k_attn_join
        const float l = half_sum(st.l);
        if (!r.live) return;
        const int64_t at = (sq.q0 + r.tok) * p.Hq + r.hq, rows = p.total_q * p.Hq;
        store_column<F32, DP>(st.o, 1.0f, p.ws + ((int64_t)blockIdx.z * rows + at) * p.D, p.D, h);
        if (h == 0) {
            float *ml = p.ws + p.nsplit * rows * p.D + ((int64_t)blockIdx.z * rows + at) * 2;
            ml[0] = st.m;
            ml[1] = l;
        }
        return;
    }
    finish_rows<E, DP>(p, sq, st, r, h);
}

// ---- joining the key ranges of a row: one wave a row (of a sequence that the tile kernel took) ----

template <class E>
__global__ void __launch_bounds__(256) k_attn_join(const AttnParams p) {
    const int lane = threadIdx.x & 63;
    const int64_t rows = p.total_q * p.Hq;
    for (int64_t at = (int64_t)blockIdx.x * 4 + uniform((int)(threadIdx.x >> 6)); at < rows; at += (int64_t)gridDim.x * 4) {
        const Joined r = join_parts((const float2 *)(p.ws + p.nsplit * rows * p.D), p.ws, at, rows, 0, 1, p.nsplit, p.D, lane);
        const int tok = (int)(at / p.Hq), hq = (int)(at - (int64_t)tok * p.Hq);
        int seq;
        const Seq sq = seq_of_row(p, tok, seq);
        const int t = tok - (int)sq.q0;
        if (t < 0 || t >= sq.lq || sq.lq * p.grp <= p.rcap) continue;
        finish_joined<E>(p, r, tok, hq, sq.lk == 0 || (p.causal && t + sq.lk < sq.lq), lane);
    }
}

template <class E, int DP, bool SHORT>
hipError_t run_fwd(const AttnParams &p0, hipStream_t s) {
    typedef FwdCfg<E, DP, SHORT> C;
    AttnParams p = p0;
    p.slots = p.total_q * p.grp / C::BM + p.B;
    p.run = run_of(p.slots, p.B);
    if (C::kLds + C::kFlags > 64 * 1024) {
        hipError_t e = hipFuncSetAttribute((const void *)k_attn_fwd<E, DP, SHORT>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                            C::kLds + C::kFlags);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_attn_fwd<E, DP, SHORT>), dim3((unsigned)xcd_grid(p.slots, p.Hkv, p.run), 1, p.nsplit), dim3(256), C::kLds + C::kFlags, s, p);
    if (p.nsplit > 1) {
        const int64_t rows = p.total_q * p.Hq;
        hipLaunchKernelGGL((k_attn_join<E>), dim3((unsigned)std::min<int64_t>((rows + 3) / 4, 1 << 20)), dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

template <class E>
hipError_t run_fwd_e(const AttnParams &p, hipStream_t s) {
    if (p.D <= 32) return run_fwd<E, 32, false>(p, s);
    if (p.D <= 64) return run_fwd<E, 64, false>(p, s);
    if constexpr (!__is_same(E, F32))
        if (p.total_k <= kShortKeys * p.B) return run_fwd<E, 128, true>(p, s);
    return run_fwd<E, 128, false>(p, s);
}

// Key ranges a launch is split into: enough workgroups for two a compute unit where the rows alone do not give them, or
// four where so many are resident at once (half types up to 64 dims; 7 sequences up to 3102, 3 heads of 40, bf16: 53 us,
// against 66 us with two), none shorter than 256 keys on average, or 64 in fp32, whose products take eight times as long
// (9 sequences up to 650, 2 heads on 1 of 32: 19 us, against 38 us with 256).
int pick_nsplit(const AttnParams &p, bool half) {
    const int64_t wgs = (p.total_q * p.grp / 128 + p.B) * p.Hkv;
    const int64_t want = (half && p.D <= 64 ? 4 : 2) * (int64_t)device_num_cus();
    const int64_t most = std::max<int64_t>(1, p.total_k / p.B / (half ? 256 : 64));
    return (int)std::min<int64_t>(std::max<int64_t>(1, want / std::max<int64_t>(1, wgs)), std::min<int64_t>(most, 64));
}

}  // namespace

size_t attention_workspace_bytes(const AttnParams &p0, eqlin_dtype_t dtype) {
    AttnParams p = p0;
    if (p.total_q <= 0 || p.B <= 0) return 0;
    const bool step = plan_step(p);
    const int n = pick_nsplit(p, dtype != EQLIN_F32);
    const size_t parts = n <= 1 || (step && !p.tiled) ? 0 : (size_t)n * p.total_q * p.Hq * (p.D + 2) * sizeof(float);
    return parts + (step ? step_workspace_bytes(p) : 0);
}

hipError_t launch_attention(const AttnParams &p0, eqlin_dtype_t dtype, hipStream_t s) {
    AttnParams p = p0;
    const bool step = plan_step(p);
    if (!step || p.tiled) {
        AttnParams t = p;
        t.nsplit = pick_nsplit(p, dtype != EQLIN_F32);
        if (step) t.ws += step_workspace_bytes(p) / sizeof(float);
        const hipError_t e = dtype == EQLIN_F32 ? run_fwd_e<F32>(t, s) : dtype == EQLIN_F16 ? run_fwd_e<F16>(t, s) : run_fwd_e<BF16>(t, s);
        if (e != hipSuccess || !step) return e;
    }
    return launch_step(p, dtype, s);
}

}  // namespace eqlin

// attn_step.hip -- attention of few query rows over many keys (a new token over a cache): the keys of a sequence
// are split into chunks, one wave takes a chunk, and the partial results are joined.
//
// Bound by reading k and v once. A workgroup is one wave: it keeps two 32-key tiles of k and v in flight straight
// into LDS (32 KB at 128 dims in a half type; the registers let four waves share a CU, 128 KB on their way), with no
// barrier and no other wave to wait for. The group's rows are the 32 columns of its products. 8 tokens over
// 100000 keys in all, 16 heads on 2 of 128 dims in bf16 (103 MB): 29.3 us with the join, 3.5 TB/s; the chunks' kernel
// alone 24 us, 4.3 TB/s, against 5.1 TB/s of a large copy. Sequences of more rows than the columns hold are the tile
// kernel's, launched before.
#include "attn.h"
#include "attn_fwd.h"

namespace eqlin {

namespace {

template <class E, int DP>
struct StepCfg {
    typedef Tile<E, DP> TL;
    static constexpr int BN = 32;
    static constexpr int kTileBytes = BN * TL::kRow;
    static constexpr int kLds = 4 * kTileBytes;
    typedef TileDma<E, DP, BN, 1> Dma;
};

// Rows of 32 (columns of the products) from packed row `row0` on over the keys [k_beg, k_end).
template <class E, int DP>
__device__ __forceinline__ void step_rows(const AttnParams &p, const Seq &sq, int hk, int row0, int k_beg, int k_end, char *lds,
                                          int lane, FwdState<E, DP> &st, Rows &r) {
    typedef StepCfg<E, DP> C;
    typedef Tile<E, DP> TL;
    typedef typename ElemOf<E>::type T;
    const int h = lane >> 5;
    const uint32_t lds0 = lds_offset(lds);
    r = rows_of(p, sq, hk, row0, 32, 0, lane);
    k_end = min(k_end, r.k_end);
    const T *kg = (const T *)p.k + sq.k0 * p.kt + hk * p.kh;
    const T *vg = (const T *)p.v + sq.k0 * p.vt + hk * p.vh;
    typename C::Dma dk, dv;
    auto fetch = [&](int k0, int buf) {
        const int valid = sq.lk - k0;
        if (valid < C::BN) {
            dk.offsets(p.kt, valid, 0, lane);
            dv.offsets(p.vt, valid, 0, lane);
        }
        dk.issue(lds0 + buf * 2 * C::kTileBytes, kg + (int64_t)k0 * p.kt, p.D, 0, lane);
        dv.issue(lds0 + buf * 2 * C::kTileBytes + C::kTileBytes, vg + (int64_t)k0 * p.vt, p.D, 0, lane);
    };
    dk.offsets(p.kt, C::BN, 0, lane);
    dv.offsets(p.vt, C::BN, 0, lane);
    uint4 qf[TL::kSteps];
    load_row<E, DP>(qf, (const T *)p.q + (sq.q0 + r.tok) * p.qt + r.hq * p.qh, p.D, h);
    if (k_beg < k_end) fetch(k_beg, 0);
    if (k_beg + C::BN < k_end) fetch(k_beg + C::BN, 1);
    st.clear();
    const float c = p.scale * kLog2e;
    const typename TL::Lane L = TL::lane_of(lane);
    int buf = 0;
    bool bad = false;  // some tile was cleared
    for (int k0 = k_beg; k0 < k_end; k0 += C::BN) {
        // whole heads: the younger tile's loads may stay on their way
        if (p.D == DP && k0 + C::BN < k_end) dma_wait_but<2 * C::Dma::N>();
        else dma_wait();
        const uint32_t kt = lds0 + buf * 2 * C::kTileBytes, vt = kt + C::kTileBytes;
        if (k0 + C::BN - 1 > r.all) {
            char *v = lds + (2 * buf + 1) * C::kTileBytes;
            if (__any(tile_nonfinite<E, 64>(v, C::kTileBytes, lane))) {
                bad = true;
                clear_nonfinite<E, 64>(v, C::kTileBytes, lane);
            }
        }
        fwd_block<E, DP, 1>(st, qf, L, kt, vt, c, k0 + C::BN - 1 > r.wave_min, r.last - k0, h);
        lds_read_wait();  // this tile's reads are done before its place is written again
        if (k0 + 2 * C::BN < k_end) fetch(k0 + 2 * C::BN, buf);
        buf ^= 1;
    }
    if (bad)  // tiles begin at k_beg + 32 i, and they were looked over from the one that holds key r.all + 1 on
        add_nonfinite<E, DP>(st.o, k_beg + max(0, r.all + 1 - k_beg) / C::BN * C::BN, min(r.wave_max, k_end - 1), p.D, h,
                             [&](int j) { return vg + (int64_t)j * p.vt; }, [&](int j) { return j <= r.last; });
}

template <class E, int DP>
__global__ void __launch_bounds__(64, DP > 64 ? 1 : 2) k_attn_step(const AttnParams p) {
    typedef StepCfg<E, DP> C;
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x, h = lane >> 5;
    const int hk = (int)(blockIdx.x % (uint32_t)p.Hkv);
    const int64_t slot = blockIdx.x / (uint32_t)p.Hkv;
    int64_t tile;
    const Seq sq = seq_of_slot<true>(p, 1, p.chunk, slot, tile);
    const int64_t k_at = tile * p.chunk;
    if (tile < 0 || k_at >= sq.lk) return;
    zero_pad<64>(lds, C::kLds, p.D, DP, lane);
    const int rows = sq.lq * p.grp, chunks = (sq.lk + p.chunk - 1) / p.chunk;
    FwdState<E, DP> st;
    Rows r;
    if (rows > p.rcap && p.tiled) return;
    // one chunk, or more rows than a partial result has room for: whole rows, shared out over the chunks' waves
    const bool split = rows <= p.rcap && chunks > 1;
    const int k_beg = split ? (int)k_at : 0, k_end = split ? (int)min(k_at + p.chunk, (int64_t)sq.lk) : sq.lk;
    for (int row0 = split ? 0 : (int)tile * 32; row0 < rows; row0 += split ? 32 : chunks * 32) {
        step_rows<E, DP>(p, sq, hk, row0, k_beg, k_end, lds, lane, st, r);
        if (split) {
            const float l = half_sum(st.l);
            if (r.live) {
                const int64_t at = (slot * p.Hkv + hk) * p.rcap + (lane & 31);
                store_column<F32, DP>(st.o, 1.0f, p.ws + at * p.D, p.D, h);
                if (h == 0) {
                    float *ml = p.ws + p.slots * p.Hkv * p.rcap * p.D + at * 2;
                    ml[0] = st.m;
                    ml[1] = l;
                }
            }
        } else {
            finish_rows<E, DP>(p, sq, st, r, h);
        }
        lds_read_wait();
    }
}

// A workgroup a sequence and head (and token, blockIdx.y): its 16 waves share the chunks, then join over LDS.
constexpr int kJoinWaves = 16;
template <class E>
__global__ void __launch_bounds__(64 * kJoinWaves) k_attn_step_join(const AttnParams p) {
    __shared__ float2 so[kJoinWaves][64], sml[kJoinWaves];
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    // (the loop over units: one turn, but for more than a million of them)
    for (int64_t unit = blockIdx.x, step_u = gridDim.x; unit < (int64_t)p.B * p.Hq; unit += step_u) {
        const int seq = (int)(unit / p.Hq), hq = (int)(unit - (int64_t)seq * p.Hq), hk = hq / p.grp;
        const Seq sq = seq_at(p, seq);
        const int nr = sq.lq * p.grp, chunks = (sq.lk + p.chunk - 1) / p.chunk;
        if (nr > p.rcap && p.tiled) continue;                      // the tile kernel's
        if (chunks == 1 || (nr > p.rcap && chunks > 0)) continue;  // written by the step itself
        for (int tok = blockIdx.y; tok < sq.lq; tok += gridDim.y) {
            const int64_t slot0 = slot_start(sq.k0, seq, 1, p.chunk);
            const int64_t base = (slot0 * p.Hkv + hk) * p.rcap + tok * p.grp + (hq - hk * p.grp), step = (int64_t)p.Hkv * p.rcap;
            const float2 *ml = (const float2 *)(p.ws + p.slots * p.Hkv * p.rcap * p.D);
            // each wave joins its own chunks (their loads wait for nothing), then the waves join
            const Joined r = join_parts(ml, p.ws, base, step, wave, kJoinWaves, chunks, p.D, lane);
            __syncthreads();
            so[wave][lane] = r.o;
            if (lane == 0) sml[wave] = make_float2(r.m, r.l);
            __syncthreads();
            if (wave == 0) {
                Joined all = {-INFINITY, 0.0f, make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int w = 0; w < kJoinWaves; ++w) all.m = fmaxf(all.m, sml[w].x);
                const float mm = all.m == -INFINITY ? 0.0f : all.m;
#pragma unroll
                for (int w = 0; w < kJoinWaves; ++w) {
                    const float a = __builtin_amdgcn_exp2f(sml[w].x - mm);
                    all.l = fmaf(a, sml[w].y, all.l);
                    all.o.x = fmaf(a, so[w][lane].x, all.o.x);
                    all.o.y = fmaf(a, so[w][lane].y, all.o.y);
                }
                finish_joined<E>(p, all, sq.q0 + tok, hq, sq.lk == 0 || (p.causal && tok + sq.lk < sq.lq), lane);
            }
        }
    }
}

template <class E, int DP>
hipError_t run_step(const AttnParams &p, hipStream_t s) {
    typedef StepCfg<E, DP> C;
    hipLaunchKernelGGL((k_attn_step<E, DP>), dim3((unsigned)(p.slots * p.Hkv)), dim3(64), C::kLds, s, p);
    const int toks = (int)std::min<int64_t>((p.total_q + p.B - 1) / p.B, std::max(1, p.rcap / p.grp));
    hipLaunchKernelGGL((k_attn_step_join<E>), dim3((unsigned)std::min<int64_t>((int64_t)p.B * p.Hq, 1 << 20), toks), dim3(64 * kJoinWaves), 0, s, p);
    return hipGetLastError();
}

template <class E>
hipError_t run_step_e(const AttnParams &p, hipStream_t s) {
    if (p.D <= 32) return run_step<E, 32>(p, s);
    if (p.D <= 64) return run_step<E, 64>(p, s);
    return run_step<E, 128>(p, s);
}

}  // namespace

bool plan_step(AttnParams &p) {
    // Few rows a sequence (they fit the 32 columns on average) over enough keys that a chunk is worth a join; or,
    // of several sequences, some may be such among others with many rows (steps and pieces of prompts in one call):
    // the keys are many times the rows then. The tile kernel takes those others, one call after the other (7 steps over
    // 32768 keys and a prompt of 512, 32 heads on 8: 212 us, against 562 us by the tile kernel alone).
    const bool few = p.total_q * p.grp <= 32 * (int64_t)p.B;
    if (p.grp > 32 || p.total_k <= 256 * (int64_t)p.B || !(few || (p.B > 1 && 8 * p.total_q <= p.total_k))) return false;
    const bool several = p.total_q > p.B;  // some sequence has more than one token
    p.tiled = several && p.total_q * p.grp > 32;  // (fewer rows in all: no sequence has more than the columns hold)
    // Sequences and heads enough to fill the card with a workgroup each are the tile kernel's alone (32 heads on 8; 256 x
    // 1024 keys: 204 us, against 288 us here; 63 steps over 8192 keys and a prompt of 400: 383 us, against 480 us), but
    // not single tokens over many keys, where chunks level out sequences of different lengths (64 of 200 to 8200 keys:
    // 224 us here, against 296 us; the price, 64 of 4096 each: 219 us, against 193 us).
    const int64_t own = (int64_t)p.B * p.Hkv;
    if (own >= 2 * (int64_t)device_num_cus() && (several || p.total_k <= 2048 * (int64_t)p.B)) return false;
    // Four waves a compute unit are resident at once (registers at 128 dims in a half type). Where a chunk a wave
    // keeps them all busy in one go, chunks have that length (8 sequences, 100000 keys in all, 2 heads: 35 us,
    // against 46 us in one and a half goes); with sequences and heads enough by themselves, a third of a
    // sequence (64 x 4096 keys, 8 heads: 219 us; when this was chosen 243 us, a half 293 us, whole sequences 257 us).
    const int64_t waves = 4 * (int64_t)device_num_cus();
    int64_t chunk = 2 * own < waves ? (p.total_k * p.Hkv + waves - own - 1) / (waves - own) : (p.total_k / p.B + 2) / 3;
    chunk = std::min<int64_t>(std::max<int64_t>((chunk + 31) / 32 * 32, 128), 1 << 20);
    p.chunk = (int)chunk;
    p.rcap = several ? 32 : p.grp;
    p.slots = p.total_k / chunk + p.B;
    return true;
}

size_t step_workspace_bytes(const AttnParams &p) { return (size_t)p.slots * p.Hkv * p.rcap * (p.D + 2) * sizeof(float); }

hipError_t launch_step(const AttnParams &p, eqlin_dtype_t dtype, hipStream_t s) {
    if (dtype == EQLIN_F32) return run_step_e<F32>(p, s);
    if (dtype == EQLIN_F16) return run_step_e<F16>(p, s);
    return run_step_e<BF16>(p, s);
}

}  // namespace eqlin

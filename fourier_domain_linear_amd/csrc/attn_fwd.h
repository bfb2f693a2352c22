// attn_fwd.h -- the running softmax over key tiles in LDS, shared by the tile kernel and the step kernel.
#pragma once

#include "attn_tile.h"

namespace eqlin {

// Running softmax state of a lane's column and its O^T accumulators.
template <class E, int DP>
struct FwdState {
    f32x16 o[DP / 32];
    float m, l;  // m: running maximum in log2 units (scaled); l: this lane's half of the sum
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int db = 0; db < DP / 32; ++db) o[db] = zero16();
        m = -INFINITY;
        l = 0.0f;
    }
};

// One tile of 32 NKB keys against a wave's 32 columns. lim: last key (within the tile) the column may see;
// masked: some key of the tile is beyond some column's lim. (The test wraps the masking alone: accumulators that
// two branches write cost a second set of registers.)
template <class E, int DP, int NKB>
__device__ __forceinline__ void fwd_block(FwdState<E, DP> &st, const uint4 *qf, const typename Tile<E, DP>::Lane &L, uint32_t kt,
                                          uint32_t vt, float c, bool masked, int lim, int h) {
    typedef Tile<E, DP> TL;
    f32x16 s[NKB];
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb) {
        s[kb] = zero16();
#pragma unroll
        for (int t = 0; t < TL::kSteps; ++t) s[kb] = mma_frag<E>(TL::row_frag(kt, L, kb, t), qf[t], s[kb]);
    }
    if constexpr (!__is_same(E, F32) && DP == 128) read_ahead<NKB * TL::kSteps, NKB * TL::kSteps, NKB == 1 ? 4 : 6>();
    if (masked) {
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
            for (int v = 0; v < 16; ++v) s[kb][v] = 32 * kb + d_row(v, 0) <= lim - 4 * h ? s[kb][v] : -INFINITY;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
        for (int v = 0; v < 16; ++v) mx = fmaxf(mx, s[kb][v]);
    mx = half_max(mx) * c;
    // The maximum is only raised when it grew by more than 8 (in log2 units): a stale one keeps every
    // p <= 2^8, exact in the sums' fp32 and in range of fp16, and saves the pass over the accumulators.
    if (__any(mx > st.m + 8.0f)) {
        const float mn = fmaxf(st.m, mx);
        const float a = st.m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - mn);  // (nothing summed yet: 1)
        st.m = mn;
        st.l *= a;
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
            for (int v = 0; v < 16; ++v) st.o[db][v] *= a;
    }
    const float mm = st.m == -INFINITY ? 0.0f : st.m;
    float sum = 0.0f;
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb) {
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            s[kb][v] = __builtin_amdgcn_exp2f(fmaf(s[kb][v], c, -mm));
            sum += s[kb][v];
        }
        WFrags<E> w;
        w.set(s[kb]);
#pragma unroll
        for (int f = 0; f < WFrags<E>::NF; ++f)
#pragma unroll
            for (int db = 0; db < DP / 32; ++db)
                st.o[db] = mma_frag<E>(TL::col_frag(vt, L, kb, f, db), w.f[f], st.o[db]);
    }
    st.l += sum;
}

// A wave's rows, normalised: o and lse.
template <class E, int DP>
__device__ __forceinline__ void finish_rows(const AttnParams &p, const Seq &sq, const FwdState<E, DP> &st, const Rows &r, int h) {
    typedef typename ElemOf<E>::type T;
    const float l = half_sum(st.l);
    const bool empty = r.last < 0;
    if (!r.live) return;
    store_column<E, DP>(st.o, empty ? 0.0f : 1.0f / l, (T *)p.o + (sq.q0 + r.tok) * p.ot + r.hq * p.oh, p.D, h);
    if (p.lse && h == 0) p.lse[(sq.q0 + r.tok) * p.Hq + r.hq] = empty ? -INFINITY : st.m * kLn2 + logf(l);
}

}  // namespace eqlin

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
    // p <= 2^8, exact in the sums' fp32 and in range of fp16, and saves the pass over the accumulators. Each column's own
    // scores decide, so that its bits depend neither on the columns beside it nor on keys that it does not see.
    if (__any(mx > st.m + 8.0f)) {
        const float mn = mx > st.m + 8.0f ? mx : st.m;
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

// ---- joining partial results: softmax sums over parts of a row's keys ----
//
// Part z of a row: (m, l) at ml[base + z step] and the D unnormalised values of o behind it at o[(base + z step) D]. A
// wave joins the parts first, first + stride, ... of n, eight at a time with all loads in flight; lane l holds the
// values 2 l and 2 l + 1.
struct Joined {
    float m, l;
    float2 o;
};
__device__ __forceinline__ Joined join_parts(const float2 *ml, const float *o, int64_t base, int64_t step, int first, int stride, int n,
                                             int D, int lane) {
    constexpr int N = 8;
    Joined r = {-INFINITY, 0.0f, make_float2(0.0f, 0.0f)};
    const bool mine = 2 * lane < D;
    for (int z0 = first; z0 < n; z0 += N * stride) {
        float2 st[N], v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int z = z0 + j * stride;
            const int64_t i = base + min(z, n - 1) * step;
            st[j] = z < n ? ml[i] : make_float2(-INFINITY, 0.0f);
            v[j] = z < n && mine ? *(const float2 *)(o + i * D + 2 * lane) : make_float2(0.0f, 0.0f);
        }
        float mn = r.m;
#pragma unroll
        for (int j = 0; j < N; ++j) mn = fmaxf(mn, st[j].x);
        const float mm = mn == -INFINITY ? 0.0f : mn, a = __builtin_amdgcn_exp2f(r.m - mm);
        r.l *= a, r.o.x *= a, r.o.y *= a;
        r.m = mn;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float w = __builtin_amdgcn_exp2f(st[j].x - mm);
            r.l = fmaf(w, st[j].y, r.l);
            r.o.x = fmaf(w, v[j].x, r.o.x);
            r.o.y = fmaf(w, v[j].y, r.o.y);
        }
    }
    return r;
}

// A joined row (head hq of query token t), normalised: o and lse.
template <class E>
__device__ __forceinline__ void finish_joined(const AttnParams &p, const Joined &r, int64_t t, int hq, bool empty, int lane) {
    typedef typename ElemOf<E>::type T;
    const float inv = empty ? 0.0f : 1.0f / r.l;
    T *dst = (T *)p.o + t * p.ot + hq * p.oh + 2 * lane;
    if (2 * lane < p.D) {
        if constexpr (__is_same(E, F32)) *(float2 *)dst = make_float2(r.o.x * inv, r.o.y * inv);
        else *(uint32_t *)dst = pack2<E>(r.o.x * inv, r.o.y * inv);
    }
    if (p.lse && lane == 0) p.lse[t * p.Hq + hq] = empty ? -INFINITY : r.m * kLn2 + logf(r.l);
}

}  // namespace eqlin

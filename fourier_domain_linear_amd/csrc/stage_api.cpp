// stage_api.cpp -- the C entry points of the operators between the layers (norm, rotary positions,
// attention): argument checks and dispatch. Nothing here computes; every step runs in the HIP kernels.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>

#include "eqlin_internal.h"

using eqlin::api_fail;

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const char *x = (const char *)a, *y = (const char *)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}
// memory of an argument, from its first byte to its last
struct Span {
    const void *at;
    size_t bytes;
    const char *name;
};
// What is written overlaps neither what is read nor other memory that is written.
template <size_t NO, size_t NI>
eqlin_status_t check_apart(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (size_t a = 0; a < NO; ++a) {
        for (const Span &in : ins)
            if (overlap(outs[a].at, outs[a].bytes, in.at, in.bytes))
                return api_fail(EQLIN_ERR_INVALID_ARG, "%s overlaps the input %s", outs[a].name, in.name);
        for (size_t b = 0; b < a; ++b)
            if (overlap(outs[a].at, outs[a].bytes, outs[b].at, outs[b].bytes))
                return api_fail(EQLIN_ERR_INVALID_ARG, "%s overlaps %s", outs[a].name, outs[b].name);
    }
    return EQLIN_OK;
}
size_t elem_bytes(eqlin_dtype_t d) { return d == EQLIN_F32 ? 4 : 2; }
bool valid_dtype(eqlin_dtype_t d) { return d == EQLIN_F32 || d == EQLIN_BF16 || d == EQLIN_F16; }
int ilog2(int g) {
    int s = 0;
    while ((1 << s) < g) ++s;
    return s;
}

eqlin_status_t done(hipError_t e, const char *what) {
    return e == hipSuccess ? EQLIN_OK : api_fail(EQLIN_ERR_HIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
}

eqlin_status_t check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need == 0) return EQLIN_OK;
    if (!ws || bytes < need) return api_fail(EQLIN_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", need, ws ? bytes : (size_t)0);
    if (!aligned(ws, 256)) return api_fail(EQLIN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    return EQLIN_OK;
}

// shared checks of the norm's entry points
eqlin_status_t check_norm(int64_t N, int C, int G, eqlin_dtype_t dtype) {
    if (N < 0) return api_fail(EQLIN_ERR_INVALID_ARG, "N = %lld < 0", (long long)N);
    if (C < 1) return api_fail(EQLIN_ERR_INVALID_ARG, "C = %d must be >= 1", C);
    if (!(G == 1 || G == 2 || G == 4 || G == 8)) return api_fail(EQLIN_ERR_INVALID_ARG, "G = %d not in {1, 2, 4, 8}", G);
    if (!valid_dtype(dtype)) return api_fail(EQLIN_ERR_INVALID_ARG, "bad dtype %d", (int)dtype);
    if ((int64_t)C * G > (1 << 20)) return api_fail(EQLIN_ERR_UNSUPPORTED, "C * G = %lld beyond 2^20", (long long)C * G);
    if (N > (INT64_C(1) << 60) / ((int64_t)C * G)) return api_fail(EQLIN_ERR_INVALID_ARG, "N = %lld overflows the index range", (long long)N);
    return EQLIN_OK;
}

eqlin_status_t rmsnorm(const void *x, const void *residual, const void *gamma, void *sum, void *y, uint8_t *q,
                       float *scale, float *rstd, int64_t N, int C, int G, float eps, eqlin_dtype_t dtype,
                       eqlin_stream_t stream, bool quant, const char *what) {
    eqlin::api_clear();
    eqlin_status_t st = check_norm(N, C, G, dtype);
    if (st != EQLIN_OK) return st;
    if (!(eps >= 0.0f) || isinf(eps)) return api_fail(EQLIN_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (N == 0) return EQLIN_OK;
    const void *out = quant ? (const void *)q : y;
    if (!x || !out || (quant && !scale)) return api_fail(EQLIN_ERR_INVALID_ARG, "null x or output");
    const size_t eb = elem_bytes(dtype), n = (size_t)N * C * G;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(sum, 16) || !aligned(out, 16))
        return api_fail(EQLIN_ERR_INVALID_ARG, "x, residual, sum and the output must be 16-byte aligned");
    if (!aligned(gamma, eb) || !aligned(rstd, 4) || !aligned(scale, 4)) return api_fail(EQLIN_ERR_INVALID_ARG, "gamma, rstd or scale misaligned");
    const size_t ob = quant ? n : n * eb;
    const Span ins[] = {{x, n * eb, "x"}, {residual, n * eb, "residual"}, {gamma, (size_t)C * eb, "gamma"}};
    const Span outs[] = {{sum, n * eb, "sum"}, {out, ob, quant ? "q" : "y"}, {rstd, (size_t)N * 4, "rstd"}, {scale, (size_t)N * 4, "scale"}};
    if ((st = check_apart(outs, ins)) != EQLIN_OK) return st;
    eqlin::NormParams p = {x, residual, gamma, sum, y, q, scale, rstd, N, C, ilog2(G), eps};
    (void)hipGetLastError();
    return done(eqlin::launch_rmsnorm(p, dtype, (hipStream_t)stream), what);
}

// a stride over n tokens or heads: of one it means nothing, whatever it is
int64_t stride_of(int64_t stride, int64_t n) { return n > 1 ? stride : 0; }

// arguments shared by the attention's entry points -> the kernels' parameters
eqlin_status_t check_attention(const eqlin_attention_args *a, eqlin::AttnParams *p) {
    if (!a) return api_fail(EQLIN_ERR_INVALID_ARG, "null arguments");
    if (!valid_dtype(a->dtype)) return api_fail(EQLIN_ERR_INVALID_ARG, "bad dtype %d", (int)a->dtype);
    if (a->batch < 0 || a->total_q < 0 || a->total_k < 0)
        return api_fail(EQLIN_ERR_INVALID_ARG, "batch = %d, total_q = %lld, total_k = %lld", a->batch, (long long)a->total_q, (long long)a->total_k);
    if (a->heads_q < 1 || a->heads_kv < 1 || a->heads_q % a->heads_kv != 0)
        return api_fail(EQLIN_ERR_INVALID_ARG, "heads_q = %d must be a multiple of heads_kv = %d", a->heads_q, a->heads_kv);
    const int per = a->dtype == EQLIN_F32 ? 4 : 8;
    if (a->dim < 1) return api_fail(EQLIN_ERR_INVALID_ARG, "dim = %d", a->dim);
    if (a->dim > 128 || a->dim % per != 0)
        return api_fail(EQLIN_ERR_UNSUPPORTED, "dim = %d: a multiple of %d up to 128", a->dim, per);
    if (!(a->scale > 0.0f) || isinf(a->scale)) return api_fail(EQLIN_ERR_INVALID_ARG, "scale must be finite and > 0");
    // the launches' index range (at most 2^24 workgroups)
    if (a->total_q > (1 << 29) / a->heads_q || a->total_k > (1 << 29) / a->heads_kv || a->batch > (1 << 21) / a->heads_kv)
        return api_fail(EQLIN_ERR_UNSUPPORTED, "total_q * heads_q or total_k * heads_kv beyond 2^29, or batch * heads_kv beyond 2^21");
    *p = eqlin::AttnParams{};
    p->q = a->q, p->k = a->k, p->v = a->v, p->o = a->o, p->lse = a->lse;
    p->qt = stride_of(a->q_token_stride, a->total_q), p->qh = stride_of(a->q_head_stride, a->heads_q);
    p->kt = stride_of(a->k_token_stride, a->total_k), p->kh = stride_of(a->k_head_stride, a->heads_kv);
    p->vt = stride_of(a->v_token_stride, a->total_k), p->vh = stride_of(a->v_head_stride, a->heads_kv);
    p->ot = stride_of(a->o_token_stride, a->total_q), p->oh = stride_of(a->o_head_stride, a->heads_q);
    p->cu_q = a->cu_q, p->cu_k = a->cu_k, p->len_k = a->len_k;
    p->total_q = a->total_q, p->total_k = a->total_k;
    p->B = a->batch, p->Hq = a->heads_q, p->Hkv = a->heads_kv, p->grp = a->heads_q / a->heads_kv, p->D = a->dim;
    p->lgrp = (p->grp & (p->grp - 1)) == 0 ? ilog2(p->grp) : -1;
    p->scale = a->scale, p->causal = a->causal != 0;
    p->nsplit = 1;
    return EQLIN_OK;
}

// a [tokens][heads][dim] tensor's pointer and strides
eqlin_status_t check_tensor(const void *t, int64_t ts, int64_t hs, int64_t tokens, int heads, eqlin_dtype_t dtype,
                            const char *name) {
    if (tokens == 0) return EQLIN_OK;
    if (!t) return api_fail(EQLIN_ERR_INVALID_ARG, "null %s", name);
    const int per = dtype == EQLIN_F32 ? 4 : 8;
    if (!aligned(t, 16) || ts % per != 0 || hs % per != 0)
        return api_fail(EQLIN_ERR_INVALID_ARG, "%s must be 16-byte aligned, its strides multiples of %d elements", name, per);
    // a tile of up to 64 rows is addressed with 32-bit byte offsets from its first
    if (ts < 0 || hs < 0) return api_fail(EQLIN_ERR_INVALID_ARG, "%s: negative strides", name);
    if (ts > (INT64_C(1) << 23) || hs > (INT64_C(1) << 28) / heads)
        return api_fail(EQLIN_ERR_UNSUPPORTED, "%s: token stride beyond 2^23 or heads beyond 2^28 elements", name);
    return EQLIN_OK;
}

// Whether heads of two tensors of one layout share elements: head j of token i is the dim elements from i ts + j hs on (and
// `by` further in the second tensor). Only differences of tokens and heads count; of the two kinds the one with fewer
// values is gone through, and the other's then lie in a range. self: the second tensor is the first.
bool heads_meet(int64_t ts, int64_t hs, int64_t dim, int64_t tokens1, int64_t heads1, int64_t tokens2, int64_t heads2, int64_t by, bool self) {
    if (tokens1 + tokens2 < heads1 + heads2) return heads_meet(hs, ts, dim, heads1, tokens1, heads2, tokens2, by, self);
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };  // b > 0
    for (int64_t j = -(heads1 - 1); j < heads2; ++j) {
        const int64_t at = by + j * hs;
        int64_t lo = -(tokens1 - 1), hi = tokens2 - 1;  // differences i with |at + i ts| < dim
        if (ts > 0) {
            lo = std::max(lo, floor_div(-dim - at, ts) + 1);
            hi = std::min(hi, -floor_div(at - dim, ts) - 1);
        } else if (at <= -dim || at >= dim) {
            continue;
        }
        if (self && j == 0 ? lo < 0 || hi > 0 : lo <= hi) return true;
    }
    return false;
}

// whether a tensor that is written folds onto itself
bool folds(int64_t ts, int64_t hs, int64_t tokens, int heads, int dim) {
    if ((heads > 1 && hs < dim) || (tokens > 1 && ts < dim)) return true;
    if (heads <= 1 || tokens <= 1 || ts >= (heads - 1) * hs + dim || hs >= (tokens - 1) * ts + dim) return false;
    return heads_meet(ts, hs, dim, tokens, heads, tokens, heads, 0, true);
}

size_t extent(int64_t ts, int64_t hs, int64_t tokens, int heads, int dim, eqlin_dtype_t d) {
    return tokens == 0 ? 0 : (size_t)((tokens - 1) * ts + (heads - 1) * hs + dim) * elem_bytes(d);
}

}  // namespace

extern "C" {

eqlin_status_t eqlin_rmsnorm(const void *x, const void *residual, const void *gamma, void *sum, void *y, float *rstd,
                             int64_t N, int C, int G, float eps, eqlin_dtype_t dtype, eqlin_stream_t stream) {
    return rmsnorm(x, residual, gamma, sum, y, nullptr, nullptr, rstd, N, C, G, eps, dtype, stream, false, "eqlin_rmsnorm launch");
}

eqlin_status_t eqlin_rmsnorm_quant(const void *x, const void *residual, const void *gamma, void *sum, uint8_t *q,
                                   float *scale, float *rstd, int64_t N, int C, int G, float eps, eqlin_dtype_t dtype,
                                   eqlin_stream_t stream) {
    return rmsnorm(x, residual, gamma, sum, nullptr, q, scale, rstd, N, C, G, eps, dtype, stream, true,
                   "eqlin_rmsnorm_quant launch");
}

size_t eqlin_rmsnorm_backward_workspace(int64_t N, int C, int G) {
    return N <= 0 || C < 1 ? 0 : eqlin::rmsnorm_backward_workspace_bytes(N, C, G);
}

eqlin_status_t eqlin_rmsnorm_backward(const void *sum, const void *gamma, const float *rstd, const void *dy,
                                      const void *dsum, void *dx, float *dgamma, int64_t N, int C, int G,
                                      eqlin_dtype_t dtype, void *workspace, size_t workspace_bytes,
                                      eqlin_stream_t stream) {
    eqlin::api_clear();
    eqlin_status_t st = check_norm(N, C, G, dtype);
    if (st != EQLIN_OK) return st;
    if (!aligned(dgamma, 4)) return api_fail(EQLIN_ERR_INVALID_ARG, "dgamma misaligned");
    if (N == 0 && !dgamma) return EQLIN_OK;
    if (N > 0) {
        if (!sum || !rstd || !dy || !dx) return api_fail(EQLIN_ERR_INVALID_ARG, "null sum, rstd, dy or dx");
        const size_t eb = elem_bytes(dtype), n = (size_t)N * C * G;
        if (!aligned(sum, 16) || !aligned(dy, 16) || !aligned(dsum, 16) || !aligned(dx, 16))
            return api_fail(EQLIN_ERR_INVALID_ARG, "sum, dy, dsum and dx must be 16-byte aligned");
        if (!aligned(gamma, eb) || !aligned(rstd, 4)) return api_fail(EQLIN_ERR_INVALID_ARG, "gamma or rstd misaligned");
        const size_t need = dgamma ? eqlin::rmsnorm_backward_workspace_bytes(N, C, G) : 0;
        st = check_workspace(workspace, workspace_bytes, need);
        if (st != EQLIN_OK) return st;
        const Span ins[] = {{sum, n * eb, "sum"}, {dy, n * eb, "dy"}, {dsum, n * eb, "dsum"}, {gamma, (size_t)C * eb, "gamma"}, {rstd, (size_t)N * 4, "rstd"}};
        const Span outs[] = {{dx, n * eb, "dx"}, {dgamma, (size_t)C * 4, "dgamma"}, {workspace, need, "workspace"}};
        if ((st = check_apart(outs, ins)) != EQLIN_OK) return st;
    }
    eqlin::NormGradParams p = {sum, gamma, dy, dsum, rstd, dx, dgamma, (float *)workspace, N, C, ilog2(G)};
    (void)hipGetLastError();
    return done(eqlin::launch_rmsnorm_backward(p, dtype, (hipStream_t)stream), "eqlin_rmsnorm_backward launch");
}

eqlin_status_t eqlin_rotary(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *y,
                            int64_t y_token_stride, int64_t y_head_stride, const int32_t *pos, int64_t N, int H, int dc,
                            int G, int axes, const int *pairs, double base, unsigned flags, eqlin_dtype_t dtype,
                            eqlin_stream_t stream) {
    eqlin::api_clear();
    if (!valid_dtype(dtype)) return api_fail(EQLIN_ERR_INVALID_ARG, "bad dtype %d", (int)dtype);
    if (N < 0 || H < 1 || dc < 1) return api_fail(EQLIN_ERR_INVALID_ARG, "N = %lld, H = %d, dc = %d", (long long)N, H, dc);
    if (!(G == 1 || G == 2 || G == 4 || G == 8)) return api_fail(EQLIN_ERR_INVALID_ARG, "G = %d not in {1, 2, 4, 8}", G);
    if (flags & ~(EQLIN_ROTARY_INVERSE | EQLIN_ROTARY_D4)) return api_fail(EQLIN_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if ((flags & EQLIN_ROTARY_D4) && G != 8) return api_fail(EQLIN_ERR_INVALID_ARG, "EQLIN_ROTARY_D4 needs G = 8 (got G = %d)", G);
    if (axes < 1 || axes > eqlin::kRotaryMaxAxes || !pairs) return api_fail(EQLIN_ERR_INVALID_ARG, "axes = %d: 1 to %d, with pairs", axes, eqlin::kRotaryMaxAxes);
    if (!(base > 0.0) || isinf(base)) return api_fail(EQLIN_ERR_INVALID_ARG, "base must be finite and > 0");
    eqlin::RotaryParams p = {};
    int64_t P = 0;
    for (int a = 0; a < axes; ++a) {
        if (pairs[a] < 0) return api_fail(EQLIN_ERR_INVALID_ARG, "pairs[%d] = %d < 0", a, pairs[a]);
        P += pairs[a];
        if (2 * P > dc) return api_fail(EQLIN_ERR_INVALID_ARG, "%lld pairs need more than dc = %d channels", (long long)P, dc);
        if (P > eqlin::kRotaryMaxPairs) return api_fail(EQLIN_ERR_UNSUPPORTED, "more than %d pairs", eqlin::kRotaryMaxPairs);
        p.end[a] = (int)P;
        for (int i = 0; i < pairs[a]; ++i) p.freq[P - pairs[a] + i] = pow(base, -(double)i / pairs[a]) / 6.283185307179586476925;
    }
    if (P < 1) return api_fail(EQLIN_ERR_INVALID_ARG, "no pairs");
    if ((int64_t)dc * G > (1 << 20) || H > (1 << 20)) return api_fail(EQLIN_ERR_UNSUPPORTED, "dc * G or H beyond 2^20");
    if (N > (INT64_C(1) << 40) / ((int64_t)dc * G)) return api_fail(EQLIN_ERR_UNSUPPORTED, "N = %lld overflows the index range", (long long)N);
    if (N == 0) return EQLIN_OK;
    if (!x || !y || !pos) return api_fail(EQLIN_ERR_INVALID_ARG, "null x, y or pos");
    const size_t eb = elem_bytes(dtype);
    if (!aligned(x, eb) || !aligned(y, eb) || !aligned(pos, 4)) return api_fail(EQLIN_ERR_INVALID_ARG, "x, y or pos misaligned");
    const int64_t D = (int64_t)dc * G, smost = INT64_C(1) << 26;
    x_token_stride = stride_of(x_token_stride, N), y_token_stride = stride_of(y_token_stride, N);
    x_head_stride = stride_of(x_head_stride, H), y_head_stride = stride_of(y_head_stride, H);
    if (x_token_stride < 0 || x_head_stride < 0 || y_token_stride < 0 || y_head_stride < 0 || x_token_stride > smost ||
        x_head_stride > smost || y_token_stride > smost || y_head_stride > smost)
        return api_fail(EQLIN_ERR_INVALID_ARG, "strides out of range");
    if (N > (INT64_C(1) << 56) / std::max<int64_t>(1, std::max(x_token_stride, y_token_stride)))
        return api_fail(EQLIN_ERR_UNSUPPORTED, "N = %lld tokens of these strides overflow the index range", (long long)N);
    if (folds(y_token_stride, y_head_stride, N, H, (int)D)) return api_fail(EQLIN_ERR_INVALID_ARG, "y's strides fold it onto itself");
    const size_t xb = extent(x_token_stride, x_head_stride, N, H, (int)D, dtype), yb = extent(y_token_stride, y_head_stride, N, H, (int)D, dtype);
    if (x == y) {
        if (x_token_stride != y_token_stride || x_head_stride != y_head_stride)
            return api_fail(EQLIN_ERR_INVALID_ARG, "in place, x and y need the same strides");
    } else if (overlap(y, yb, x, xb)) {
        return api_fail(EQLIN_ERR_INVALID_ARG, "x and y overlap");
    }
    if (overlap(y, yb, pos, (size_t)N * axes * 4)) return api_fail(EQLIN_ERR_INVALID_ARG, "y overlaps pos");
    p.x = x, p.y = y, p.pos = pos;
    p.N = N, p.xt = x_token_stride, p.xh = x_head_stride, p.yt = y_token_stride, p.yh = y_head_stride;
    p.H = H, p.dc = dc, p.lg = ilog2(G), p.axes = axes, p.P = (int)P;
    p.d4 = (flags & EQLIN_ROTARY_D4) != 0, p.inverse = (flags & EQLIN_ROTARY_INVERSE) != 0;
    (void)hipGetLastError();
    return done(eqlin::launch_rotary(p, dtype, (hipStream_t)stream), "eqlin_rotary launch");
}

size_t eqlin_attention_workspace(const eqlin_attention_args *a) {
    eqlin::AttnParams p;
    if (check_attention(a, &p) != EQLIN_OK) return 0;
    return eqlin::attention_workspace_bytes(p, a->dtype);
}

eqlin_status_t eqlin_attention(const eqlin_attention_args *a, void *workspace, size_t workspace_bytes,
                               eqlin_stream_t stream) {
    eqlin::api_clear();
    eqlin::AttnParams p;
    eqlin_status_t st = check_attention(a, &p);
    if (st != EQLIN_OK) return st;
    if (a->total_q == 0 || a->batch == 0) return EQLIN_OK;
    if ((st = check_tensor(a->q, p.qt, p.qh, a->total_q, p.Hq, a->dtype, "q")) != EQLIN_OK) return st;
    if ((st = check_tensor(a->k, p.kt, p.kh, a->total_k, p.Hkv, a->dtype, "k")) != EQLIN_OK) return st;
    if ((st = check_tensor(a->v, p.vt, p.vh, a->total_k, p.Hkv, a->dtype, "v")) != EQLIN_OK) return st;
    if ((st = check_tensor(a->o, p.ot, p.oh, a->total_q, p.Hq, a->dtype, "o")) != EQLIN_OK) return st;
    if (folds(p.ot, p.oh, a->total_q, p.Hq, p.D)) return api_fail(EQLIN_ERR_INVALID_ARG, "o's strides fold it onto itself");
    if (!a->cu_q || !a->cu_k) return api_fail(EQLIN_ERR_INVALID_ARG, "null cu_q or cu_k");
    if (!aligned(a->cu_q, 4) || !aligned(a->cu_k, 4) || !aligned(a->len_k, 4) || !aligned(a->lse, 4))
        return api_fail(EQLIN_ERR_INVALID_ARG, "cu_q, cu_k, len_k or lse misaligned");
    const size_t need = eqlin::attention_workspace_bytes(p, a->dtype), cu = ((size_t)a->batch + 1) * 4;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != EQLIN_OK) return st;
    const Span ins[] = {{a->q, extent(p.qt, p.qh, a->total_q, p.Hq, p.D, a->dtype), "q"}, {a->k, extent(p.kt, p.kh, a->total_k, p.Hkv, p.D, a->dtype), "k"},
                        {a->v, extent(p.vt, p.vh, a->total_k, p.Hkv, p.D, a->dtype), "v"}, {a->cu_q, cu, "cu_q"}, {a->cu_k, cu, "cu_k"},
                        {a->len_k, cu - 4, "len_k"}};
    const Span outs[] = {{a->o, extent(p.ot, p.oh, a->total_q, p.Hq, p.D, a->dtype), "o"}, {a->lse, (size_t)a->total_q * p.Hq * 4, "lse"},
                         {workspace, need, "workspace"}};
    if ((st = check_apart(outs, ins)) != EQLIN_OK) return st;
    p.ws = (float *)workspace;
    (void)hipGetLastError();
    return done(eqlin::launch_attention(p, a->dtype, (hipStream_t)stream), "eqlin_attention launch");
}

size_t eqlin_attention_backward_workspace(const eqlin_attention_args *a) {
    eqlin::AttnParams p;
    if (check_attention(a, &p) != EQLIN_OK) return 0;
    return eqlin::attention_backward_workspace_bytes(p, a->dtype);
}

eqlin_status_t eqlin_attention_backward(const eqlin_attention_args *a, const eqlin_attention_grads *g, void *workspace,
                                        size_t workspace_bytes, eqlin_stream_t stream) {
    eqlin::api_clear();
    eqlin::AttnParams p;
    eqlin_status_t st = check_attention(a, &p);
    if (st != EQLIN_OK) return st;
    if (!g) return api_fail(EQLIN_ERR_INVALID_ARG, "null gradients");
    if (a->batch == 0 || (a->total_q == 0 && a->total_k == 0)) return EQLIN_OK;
    p.dot = stride_of(g->do_token_stride, a->total_q), p.doh = stride_of(g->do_head_stride, p.Hq);
    p.dqt = stride_of(g->dq_token_stride, a->total_q), p.dqh = stride_of(g->dq_head_stride, p.Hq);
    p.dkt = stride_of(g->dk_token_stride, a->total_k), p.dkh = stride_of(g->dk_head_stride, p.Hkv);
    p.dvt = stride_of(g->dv_token_stride, a->total_k), p.dvh = stride_of(g->dv_head_stride, p.Hkv);
    struct {
        const void *t;
        int64_t ts, hs, tokens;
        int heads;
        const char *name;
        bool out;
    } t[] = {{a->q, p.qt, p.qh, a->total_q, p.Hq, "q", false},
             {a->k, p.kt, p.kh, a->total_k, p.Hkv, "k", false},
             {a->v, p.vt, p.vh, a->total_k, p.Hkv, "v", false},
             {a->o, p.ot, p.oh, a->total_q, p.Hq, "o", false},
             {g->d_o, p.dot, p.doh, a->total_q, p.Hq, "d_o", false},
             {g->dq, p.dqt, p.dqh, a->total_q, p.Hq, "dq", true},
             {g->dk, p.dkt, p.dkh, a->total_k, p.Hkv, "dk", true},
             {g->dv, p.dvt, p.dvh, a->total_k, p.Hkv, "dv", true}};
    for (const auto &x : t) {
        if ((st = check_tensor(x.t, x.ts, x.hs, x.tokens, x.heads, a->dtype, x.name)) != EQLIN_OK) return st;
        if (x.out && folds(x.ts, x.hs, x.tokens, x.heads, p.D))
            return api_fail(EQLIN_ERR_INVALID_ARG, "%s's strides fold it onto itself", x.name);
    }
    if (!a->cu_q || !a->cu_k || (a->total_q > 0 && !a->lse)) return api_fail(EQLIN_ERR_INVALID_ARG, "null cu_q, cu_k or lse");
    if (!aligned(a->cu_q, 4) || !aligned(a->cu_k, 4) || !aligned(a->len_k, 4) || !aligned(a->lse, 4))
        return api_fail(EQLIN_ERR_INVALID_ARG, "cu_q, cu_k, len_k or lse misaligned");
    const size_t need = eqlin::attention_backward_workspace_bytes(p, a->dtype), cu = ((size_t)a->batch + 1) * 4;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != EQLIN_OK) return st;
    const Span ws[] = {{workspace, need, "workspace"}};
    const Span more[] = {{a->lse, (size_t)a->total_q * p.Hq * 4, "lse"}, {a->cu_q, cu, "cu_q"}, {a->cu_k, cu, "cu_k"}, {a->len_k, cu - 4, "len_k"}};
    if ((st = check_apart(ws, more)) != EQLIN_OK) return st;
    // dq, dk and dv may be interleaved parts of one tensor (the gradient of a qkv layer's output): of two outputs only
    // shared elements are refused, which strides that differ do not tell in general
    for (const auto &x : t) {
        const Span sx[] = {{x.t, extent(x.ts, x.hs, x.tokens, x.heads, p.D, a->dtype), x.name}};
        if ((st = check_apart(ws, sx)) != EQLIN_OK) return st;
        if (!x.out) continue;
        if ((st = check_apart(sx, more)) != EQLIN_OK) return st;
        for (const auto &y : t) {
            const Span sy[] = {{y.t, extent(y.ts, y.hs, y.tokens, y.heads, p.D, a->dtype), y.name}};
            if (!y.out) {
                if ((st = check_apart(sx, sy)) != EQLIN_OK) return st;
            } else if (&x < &y && overlap(x.t, sx[0].bytes, y.t, sy[0].bytes)) {
                const int64_t by = ((const char *)y.t - (const char *)x.t) / (int64_t)elem_bytes(a->dtype);
                const int64_t ts = x.tokens > 1 ? x.ts : y.ts, hs = x.heads > 1 ? x.hs : y.hs;
                const bool alike = (y.tokens == 1 || ts == y.ts) && (y.heads == 1 || hs == y.hs);
                if (by == 0 || (alike && heads_meet(ts, hs, p.D, x.tokens, x.heads, y.tokens, y.heads, by, false)))
                    return api_fail(EQLIN_ERR_INVALID_ARG, "%s and %s share memory", x.name, y.name);
            }
        }
    }
    p.dout = g->d_o, p.dq = g->dq, p.dk = g->dk, p.dv = g->dv;
    p.ws = (float *)workspace;
    (void)hipGetLastError();
    return done(eqlin::launch_attention_backward(p, a->dtype, (hipStream_t)stream), "eqlin_attention_backward launch");
}

}  // extern "C"

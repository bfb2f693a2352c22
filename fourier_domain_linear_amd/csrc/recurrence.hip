// recurrence.hip -- gated linear recurrence over packed sequences, forward and gradients. For every sequence and every
// column (channel and group element), over the tokens in order (reverse: from the last to the first):
//
//   f = sigmoid(forget);  h_t = f_t h_{t-1} + (1 - f_t) x_t;  y_t = h_t, or h_t silu(gate_t)
//
// A stretch of tokens maps the state before it to the state after it by h -> A h + B, A = product of its f; two
// stretches in a row compose to (A' A, A' B + B'). A workgroup takes rounds of kChunk tokens by a strip of columns: each of its waves
// holds TW tokens in registers (lanes over columns, so that every load is one stretch of memory), composes them to
// (A, B), and after one exchange through LDS knows the state in front of its tokens and goes over them again,
// from the registers, for the results: x, forget and gate are read once, y is written once.
//
// The launch takes one of two forms. SEQ: a workgroup goes through a sequence, round after round. Where that leaves too
// few workgroups or too long a way (few long sequences), three launches: ENDS composes each chunk of kChunk tokens but a
// sequence's last, JOIN goes over each sequence's chunks for the states in front of them, CHUNK does the rounds side by
// side. (x and forget are then read twice, the second time mostly from the last cache.)
//
// Everything is held in fp32; 1 - f is computed as sigmoid(-forget), without the cancellation; results are rounded once.
// Sequences never meet in a workgroup's sums, so what is not finite in one has no part in another.
#include "stage.h"

namespace eqlin {

namespace {

constexpr int kChunk = kRecurrenceChunk;  // tokens of a round, of a chunk and of the distance between marks
enum Mode { SEQ, CHUNK, ENDS };

// sigmoid(z) and 1 - sigmoid(z), both to a few units of fp32's last place (half types: the hardware's exponential of
// the product with log2 e, relative error up to |z| 2^-24, far below their rounding)
template <class E>
__device__ __forceinline__ void sigmoid(float z, float &f, float &rest) {
    const float e = __is_same(E, F32) ? expf(-fabsf(z)) : __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(z));
    const float r = __builtin_amdgcn_rcpf(1.0f + e), s = e * r;
    f = z >= 0.0f ? r : s;
    rest = z >= 0.0f ? s : r;
}

// Sequence i: its first token, its length, and its first slot. Sequence i owns the chunk slots from cu[i] / kChunk + i on, at
// least as many as it has chunks, so the launch needs no lengths on the host. Bounds are forced into the tensors
// whatever the array holds.
struct Seq {
    int t0, len;
    int64_t slot;
};
__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }
__device__ __forceinline__ Seq seq_at(const RecurrenceParams &p, int i) {
    Seq s;
    s.t0 = clampi(p.cu[i], 0, (int)p.T);
    s.len = clampi(p.cu[i + 1], s.t0, (int)p.T) - s.t0;
    s.slot = s.t0 / kChunk + (int64_t)i;
    return s;
}
// The sequence that owns a slot (the last that begins at or before it), by a 64-way search of the wave.
__device__ __forceinline__ int seq_of_slot(const RecurrenceParams &p, int64_t slot) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = p.B;
    while (n > 1) {
        const int step = (n + 63) / 64, i = min(lo + lane * step, p.B - 1);
        const bool in = lane * step < n && clampi(p.cu[i], 0, (int)p.T) / kChunk + (int64_t)i <= slot;
        const int c = max(1, __popcll(__ballot(in))), skip = (c - 1) * step;
        lo += skip;
        n = min(n - skip, step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// What a workgroup works on: a strip of columns of a sequence (SEQ), or of one chunk of it.
struct Unit {
    Seq s;
    int i, tile, col;  // col: the lane's first column
    bool none;         // a slot without a chunk
};
template <Mode MODE, int EC>
__device__ __forceinline__ Unit unit_at(const RecurrenceParams &p, int64_t unit, int strips) {
    Unit u;
    const int64_t id = unit / strips;
    u.col = ((int)(unit - id * strips) * 64 + (threadIdx.x & 63)) * EC;
    u.i = MODE == SEQ ? (int)id : seq_of_slot(p, id);
    u.s = seq_at(p, u.i);
    u.tile = MODE == SEQ ? 0 : (int)(id - u.s.slot);
    u.none = u.tile < 0 || (u.tile > 0 && u.tile > (u.s.len - 1) / kChunk) || (MODE != SEQ && u.s.len == 0);
    return u;
}

// Token `at` of a sequence in the recurrence's order, the last one for what is past the end -> its place in a tensor.
__device__ __forceinline__ int64_t place(const RecurrenceParams &p, const Seq &s, int at) {
    at = min(at, s.len - 1);
    return p.reverse ? s.t0 + s.len - 1 - at : s.t0 + at;
}
template <class E, int EC>
__device__ __forceinline__ void load_tokens(const RecurrenceParams &p, const Seq &s, const void *t, int64_t stride, int at, int col,
                                            Pack<E, EC> *v, int n) {
    typedef typename Elem<E>::T T;
#pragma unroll
    for (int k = 0; k < n; ++k) v[k].load((const T *)t + place(p, s, at + k) * stride + col);
}
template <int EC>
__device__ __forceinline__ void load_state(const float *t, int64_t row, int L, int col, float *h) {
    const float *a = t + row * L + col;
    if constexpr (EC == 2) {
        const float2 v = *(const float2 *)a;
        h[0] = v.x, h[1] = v.y;
    } else {
#pragma unroll
        for (int j = 0; j < EC; ++j) h[j] = a[j];
    }
}
template <int EC>
__device__ __forceinline__ void store_state(float *t, int64_t row, int L, int col, const float *h) {
    float *a = t + row * L + col;
    if constexpr (EC == 2) {
        *(float2 *)a = make_float2(h[0], h[1]);
    } else {
#pragma unroll
        for (int j = 0; j < EC; ++j) a[j] = h[j];
    }
}

template <class E, int EC, int TW, int W, bool GATE, Mode MODE>
__global__ void __launch_bounds__(64 * W) k_recurrence(const RecurrenceParams p, int strips, int64_t units) {
    typedef typename Elem<E>::T T;
    typedef Pack<E, EC> PK;
    constexpr int ROUND = TW * W;
    static_assert(MODE == SEQ ? kChunk % ROUND == 0 : ROUND == kChunk, "marks lie between rounds");
    __shared__ float ends[2][2][W][64 * EC];  // two rounds' (A, B) of each wave
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), L = p.C << p.lg;
    int buf = 0;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const Unit u = unit_at<MODE, EC>(p, unit, strips);
        const bool in = u.col < L;
        const int col = in ? u.col : 0;
        const int first = u.tile * kChunk, past = MODE == SEQ ? u.s.len : min(u.s.len, first + kChunk);
        if (u.none || (MODE == ENDS && first + kChunk >= u.s.len)) continue;  // (nothing asks for a last chunk's end)
        float carry[EC], own[EC];  // the state in front of the round; what wave 0 adds to its stretch
#pragma unroll
        for (int j = 0; j < EC; ++j) carry[j] = own[j] = 0.0f;
        if constexpr (MODE == SEQ) {
            // The initial state is read by wave 0 alone, which hands it on in its stretch's B: it also writes the final one, so
            // the two may be one buffer.
            if (wave == 0 && p.state) load_state<EC>(p.state, u.i, L, col, own);
            if (u.s.len == 0) {
                if (wave == 0 && in && p.final) store_state<EC>(p.final, u.i, L, col, own);
                continue;
            }
        }
        if (MODE == CHUNK) load_state<EC>(p.carry, u.s.slot + u.tile, L, col, carry);
        for (int at = first; at < past; at += ROUND, buf ^= 1) {
            const int t = at + wave * TW;
            float f[TW][EC], b[TW][EC];
            PK o[GATE && MODE != ENDS ? TW : 1];
            float A[EC], B[EC];
#pragma unroll
            for (int j = 0; j < EC; ++j) A[j] = 1.0f, B[j] = own[j];
            const bool work = t < past;
            if (work) {
                PK x[TW], z[TW];
                load_tokens<E, EC>(p, u.s, p.f, p.ft, t, col, z, TW);
                load_tokens<E, EC>(p, u.s, p.x, p.xt, t, col, x, TW);
                if constexpr (GATE && MODE != ENDS) load_tokens<E, EC>(p, u.s, p.o, p.ot, t, col, o, TW);
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    float v[EC], w[EC];
                    x[k].unpack(v);
                    z[k].unpack(w);
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        float rest;
                        sigmoid<E>(w[j], f[k][j], rest);
                        b[k][j] = rest * v[j];
                        if (t + k >= past) f[k][j] = 1.0f, b[k][j] = 0.0f;
                        A[j] *= f[k][j];
                        B[j] = fmaf(f[k][j], B[j], b[k][j]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < EC; ++j) ends[buf][0][wave][lane * EC + j] = A[j], ends[buf][1][wave][lane * EC + j] = B[j];
            __syncthreads();
            float h[EC], a[EC];
#pragma unroll
            for (int j = 0; j < EC; ++j) h[j] = own[j], a[j] = 1.0f;
            if (MODE == SEQ && p.marks && wave == 0 && at % kChunk == 0 && in) {
                float m[EC];
#pragma unroll
                for (int j = 0; j < EC; ++j) m[j] = carry[j] + own[j];
                store_state<EC>(p.marks, u.s.slot + at / kChunk, L, col, m);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w == wave)
#pragma unroll
                    for (int j = 0; j < EC; ++j) h[j] += carry[j];
#pragma unroll
                for (int j = 0; j < EC; ++j) {
                    const float aw = ends[buf][0][w][lane * EC + j];
                    carry[j] = fmaf(aw, carry[j], ends[buf][1][w][lane * EC + j]);
                    if (MODE == ENDS) a[j] *= aw;
                }
            }
#pragma unroll
            for (int j = 0; j < EC; ++j) own[j] = 0.0f;
            if constexpr (MODE == ENDS) {
                if (wave == 0 && in) {
                    store_state<EC>(p.ends_a, u.s.slot + u.tile, L, col, a);
                    store_state<EC>(p.ends_b, u.s.slot + u.tile, L, col, carry);
                }
            } else if (work) {
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    float y[EC];
#pragma unroll
                    for (int j = 0; j < EC; ++j) y[j] = h[j] = fmaf(f[k][j], h[j], b[k][j]);
                    if constexpr (GATE) {
                        float g[EC];
                        o[k].unpack(g);
#pragma unroll
                        for (int j = 0; j < EC; ++j) {
                            float s, rest;
                            sigmoid<E>(g[j], s, rest);
                            y[j] *= g[j] * s;
                        }
                    }
                    if (in && t + k < past) PK::store((T *)p.y + place(p, u.s, t + k) * p.yt + col, y);
                }
            }
        }
        // the state after the last token (CHUNK: its chunk's workgroup has it)
        if (MODE != ENDS && past == u.s.len && wave == 0 && in && p.final) store_state<EC>(p.final, u.i, L, col, carry);
    }
}

// ---- gradients ----
//
//   dh_t = dy_t silu(gate_t) + f_{t+1} dh_{t+1} (+ dfinal at the last token)
//   dx = (1 - f) dh;  dforget = dh (h_{t-1} - x) f (1 - f);  dgate = dy h silu'(gate);  dstate = f_1 dh_1
//
// What goes back over a stretch's start, g_t = f_t dh_t, is composed from the last token on with the same A:
// g -> A g + B'. The states come again from x and forget, exactly as the forward had them, from its marks: the states in
// front of each chunk of kChunk tokens. SEQ and ENDS, JOIN, CHUNK as above, the chunks taken from the last to the first.
template <class E, int EC, int TW, int W, bool GATE, Mode MODE>
__global__ void __launch_bounds__(64 * W) k_recurrence_bwd(const RecurrenceParams p, int strips, int64_t units) {
    typedef typename Elem<E>::T T;
    typedef Pack<E, EC> PK;
    static_assert(TW * W == kChunk, "a round lies between marks");
    __shared__ float ends[2][3][W][64 * EC];  // two rounds' A, B and B' of each wave
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), L = p.C << p.lg;
    int buf = 0;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const Unit u = unit_at<MODE, EC>(p, unit, strips);
        const bool in = u.col < L;
        const int col = in ? u.col : 0;
        const int first = MODE == SEQ ? (u.s.len - 1) / kChunk * kChunk : u.tile * kChunk;
        if (u.none || (MODE == ENDS && u.tile == 0)) continue;  // (nothing asks what leaves the first chunk)
        float g[EC];  // what comes back from behind the round
#pragma unroll
        for (int j = 0; j < EC; ++j) g[j] = 0.0f;
        if (MODE == SEQ && p.dfinal) load_state<EC>(p.dfinal, u.i, L, col, g);
        if (MODE == CHUNK) load_state<EC>(p.carry, u.s.slot + u.tile, L, col, g);
        if (MODE == SEQ && u.s.len == 0) {
            if (wave == 0 && in && p.dstate) store_state<EC>(p.dstate, u.i, L, col, g);
            continue;
        }
        for (int at = first; at >= (MODE == SEQ ? 0 : first); at -= kChunk, buf ^= 1) {
            const int t = at + wave * TW, past = min(u.s.len, at + kChunk);
            PK x[TW], o[GATE ? TW : 1], dy[TW];
            float f[TW][EC], rest[TW][EC], d[TW][EC];
            float A[EC], B[EC], R[EC], mark[EC];
#pragma unroll
            for (int j = 0; j < EC; ++j) A[j] = 1.0f, B[j] = R[j] = 0.0f;
            if (MODE != ENDS) load_state<EC>(p.marks, u.s.slot + at / kChunk, L, col, mark);
            const bool work = t < past;
            if (work) {
                PK z[TW];
                load_tokens<E, EC>(p, u.s, p.f, p.ft, t, col, z, TW);
                load_tokens<E, EC>(p, u.s, p.dy, p.dyt, t, col, dy, TW);
                if constexpr (GATE) load_tokens<E, EC>(p, u.s, p.o, p.ot, t, col, o, TW);
                if constexpr (MODE != ENDS) load_tokens<E, EC>(p, u.s, p.x, p.xt, t, col, x, TW);
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    float v[EC], w[EC], s[EC];
                    z[k].unpack(w);
                    dy[k].unpack(d[k]);
                    if constexpr (GATE) o[k].unpack(s);
                    if constexpr (MODE != ENDS) x[k].unpack(v);
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        sigmoid<E>(w[j], f[k][j], rest[k][j]);
                        if constexpr (GATE) {
                            float sig, other;
                            sigmoid<E>(s[j], sig, other);
                            d[k][j] *= s[j] * sig;
                        }
                        if (t + k >= past) f[k][j] = 1.0f, rest[k][j] = d[k][j] = 0.0f;
                        A[j] *= f[k][j];
                        if constexpr (MODE != ENDS) B[j] = fmaf(f[k][j], B[j], t + k < past ? rest[k][j] * v[j] : 0.0f);
                    }
                }
#pragma unroll
                for (int k = TW - 1; k >= 0; --k)
#pragma unroll
                    for (int j = 0; j < EC; ++j) R[j] = f[k][j] * (d[k][j] + R[j]);
            }
#pragma unroll
            for (int j = 0; j < EC; ++j)
                ends[buf][0][wave][lane * EC + j] = A[j], ends[buf][1][wave][lane * EC + j] = B[j], ends[buf][2][wave][lane * EC + j] = R[j];
            __syncthreads();
            float h[EC], a[EC], back[EC];
#pragma unroll
            for (int j = 0; j < EC; ++j) h[j] = MODE == ENDS ? 0.0f : mark[j], a[j] = 1.0f, back[j] = 0.0f;
            if constexpr (MODE != ENDS)
#pragma unroll
                for (int w = 0; w < W - 1; ++w)
                    if (w < wave)
#pragma unroll
                        for (int j = 0; j < EC; ++j) h[j] = fmaf(ends[buf][0][w][lane * EC + j], h[j], ends[buf][1][w][lane * EC + j]);
#pragma unroll
            for (int w = W - 1; w >= 0; --w)
#pragma unroll
                for (int j = 0; j < EC; ++j) {
                    if (w == wave) back[j] = g[j];
                    const float aw = ends[buf][0][w][lane * EC + j];
                    g[j] = fmaf(aw, g[j], ends[buf][2][w][lane * EC + j]);
                    if (MODE == ENDS) a[j] *= aw;
                }
            if constexpr (MODE == ENDS) {
                if (wave == 0 && in) {
                    store_state<EC>(p.ends_a, u.s.slot + u.tile, L, col, a);
                    store_state<EC>(p.ends_b, u.s.slot + u.tile, L, col, g);
                }
            } else if (work) {
                float before[TW][EC];
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    float v[EC], w[EC], s[EC];
                    x[k].unpack(v);
                    if constexpr (GATE) o[k].unpack(s), dy[k].unpack(w);
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        before[k][j] = h[j] - v[j];
                        h[j] = fmaf(f[k][j], h[j], rest[k][j] * v[j]);
                        if constexpr (GATE) {
                            float sig, other;
                            sigmoid<E>(s[j], sig, other);
                            w[j] = w[j] * h[j] * sig * fmaf(s[j], other, 1.0f);
                        }
                    }
                    if constexpr (GATE)
                        if (p.dgo && in && t + k < past) PK::store((T *)p.dgo + place(p, u.s, t + k) * p.dgot + col, w);
                }
#pragma unroll
                for (int k = TW - 1; k >= 0; --k) {
                    float v[EC], w[EC];
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        const float dh = d[k][j] + back[j];
                        back[j] = f[k][j] * dh;
                        v[j] = rest[k][j] * dh;
                        w[j] = v[j] * before[k][j] * f[k][j];
                    }
                    if (in && t + k < past) {
                        const int64_t row = place(p, u.s, t + k);
                        PK::store((T *)p.dx + row * p.dxt + col, v);
                        PK::store((T *)p.df + row * p.dft + col, w);
                    }
                }
            }
        }
        if (MODE != ENDS && (MODE == SEQ || u.tile == 0) && wave == 0 && in && p.dstate) store_state<EC>(p.dstate, u.i, L, col, g);
    }
}

// JOIN: the states in front of a sequence's chunks, carry[0] = state, carry[c + 1] = A_c carry[c] + B_c (BACK: what comes
// back from behind them, from the last, dfinal, to the first). 64 columns a workgroup; its 16 waves share the chunks, each
// composes its stretch of them, and after one exchange goes over it again.
template <bool BACK>
__global__ void __launch_bounds__(1024) k_recurrence_join(const RecurrenceParams p, int strips, int64_t units) {
    constexpr int W = 16;
    __shared__ float ends[2][W][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), L = p.C << p.lg;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int i = (int)(unit / strips), u = (int)(unit - (int64_t)i * strips) * 64 + lane, col = u < L ? u : 0;
        const Seq s = seq_at(p, i);
        const int n = (s.len + kChunk - 1) / kChunk - 1;  // stretches between carries
        const float *from = BACK ? p.dfinal : p.state;
        float h = from ? from[(int64_t)i * L + col] : 0.0f;
        if (n < 0) {
            float *to = BACK ? p.dstate : p.final;
            if (wave == 0 && u < L && to) to[(int64_t)i * L + col] = h;
            continue;
        }
        const int share = (n + W - 1) / W, c0 = min(n, wave * share), c1 = min(n, c0 + share);
        // stretch c composes the c-th chunk in the order of the recurrence's (or the gradient's) way
        auto slot = [&](int c) { return (s.slot + (BACK ? n - c : c)) * L + col; };
        float A = 1.0f, B = 0.0f;
#pragma unroll 8
        for (int c = c0; c < c1; ++c) {
            const float a = p.ends_a[slot(c)], b = p.ends_b[slot(c)];
            A *= a;
            B = fmaf(a, B, b);
        }
        ends[0][wave][lane] = A, ends[1][wave][lane] = B;
        __syncthreads();
        if (wave == 0 && u < L) p.carry[slot(0)] = h;
        for (int w = 0; w < wave; ++w) h = fmaf(ends[0][w][lane], h, ends[1][w][lane]);
#pragma unroll 8
        for (int c = c0; c < c1; ++c) {
            h = fmaf(p.ends_a[slot(c)], h, p.ends_b[slot(c)]);
            if (u < L) p.carry[slot(c + 1)] = h;
        }
        __syncthreads();  // the exchange is used again
    }
}

constexpr int kGrid = 1 << 20;  // workgroups of a launch at most; they take further units in turn

// Columns a lane: two where pointers, strides and the width allow, so that a wave's load is 256 bytes (fp32: 512).
template <class E>
bool in_pairs(const RecurrenceParams &p, bool back) {
    const size_t size = 2 * sizeof(typename Elem<E>::T);
    auto fine = [&](const void *t, int64_t stride) { return (uintptr_t)t % size == 0 && stride % 2 == 0; };
    auto even = [&](const void *t) { return (uintptr_t)t % 8 == 0; };
    bool ok = (p.C << p.lg) % 2 == 0 && fine(p.x, p.xt) && fine(p.f, p.ft) && (!p.o || fine(p.o, p.ot)) && even(p.marks);
    if (back)
        return ok && fine(p.dy, p.dyt) && fine(p.dx, p.dxt) && fine(p.df, p.dft) && (!p.dgo || fine(p.dgo, p.dgot)) && even(p.dfinal) && even(p.dstate);
    return ok && fine(p.y, p.yt) && even(p.state) && even(p.final);
}

template <class E, int EC, bool GATE>
hipError_t run(const RecurrenceParams &p, bool back, hipStream_t s) {
    const int64_t L = (int64_t)p.C << p.lg;
    const int strips = (int)((L + 64 * EC - 1) / (64 * EC)), joins = (int)((L + 63) / 64);
    const int64_t seqs = (int64_t)p.B * strips, chunks = p.slots * strips, joined = (int64_t)p.B * joins;
    auto grid = [](int64_t units) { return dim3((unsigned)std::min<int64_t>(units, kGrid)); };
#define EQLIN_RECURRENCE(K, TW, W, G, MODE, UNITS) \
    hipLaunchKernelGGL((K<E, EC, TW, W, G, MODE>), grid(UNITS), dim3(64 * W), 0, s, p, strips, UNITS)
    if (!p.split) {
        if (back) EQLIN_RECURRENCE(k_recurrence_bwd, 16, 8, GATE, SEQ, seqs);
        else if (p.longest <= 16) EQLIN_RECURRENCE(k_recurrence, 16, 1, GATE, SEQ, seqs);
        else EQLIN_RECURRENCE(k_recurrence, 16, 8, GATE, SEQ, seqs);
        return hipGetLastError();
    }
    if (back) {
        EQLIN_RECURRENCE(k_recurrence_bwd, 16, 8, GATE, ENDS, chunks);
        hipLaunchKernelGGL(k_recurrence_join<true>, grid(joined), dim3(1024), 0, s, p, joins, joined);
        EQLIN_RECURRENCE(k_recurrence_bwd, 16, 8, GATE, CHUNK, chunks);
    } else {
        EQLIN_RECURRENCE(k_recurrence, 16, 8, false, ENDS, chunks);
        hipLaunchKernelGGL(k_recurrence_join<false>, grid(joined), dim3(1024), 0, s, p, joins, joined);
        EQLIN_RECURRENCE(k_recurrence, 16, 8, GATE, CHUNK, chunks);
    }
#undef EQLIN_RECURRENCE
    return hipGetLastError();
}

template <class E>
hipError_t run_type(const RecurrenceParams &p, bool back, hipStream_t s) {
    if (in_pairs<E>(p, back)) return p.o ? run<E, 2, true>(p, back, s) : run<E, 2, false>(p, back, s);
    return p.o ? run<E, 1, true>(p, back, s) : run<E, 1, false>(p, back, s);
}

}  // namespace

void plan_recurrence(RecurrenceParams &p) {
    const int64_t L = (int64_t)p.C << p.lg;
    p.slots = p.T / kChunk + p.B;
    const int64_t strips = (L + 127) / 128, rounds = (p.longest + kChunk - 1) / kChunk;
    // SEQ: the longest sequence's rounds one after the other, about 2 us each, or all units over the card; the three
    // launches take about 8 us more than their rounds
    p.split = rounds > 4 && rounds > 4 * (p.slots * strips / (2 * device_num_cus()));
}

// A and B (or B'), and the carries (the forward's are the marks where those are kept)
size_t recurrence_workspace_bytes(const RecurrenceParams &p) {
    return p.split ? 3 * (size_t)p.slots * ((size_t)p.C << p.lg) * sizeof(float) : 0;
}

hipError_t launch_recurrence(RecurrenceParams p, eqlin_dtype_t dtype, bool back, float *ws, hipStream_t s) {
    if (p.split) {
        const size_t states = (size_t)p.slots * ((size_t)p.C << p.lg);
        p.ends_a = ws, p.ends_b = ws + states;
        p.carry = back || !p.marks ? ws + 2 * states : p.marks;
    }
    if (dtype == EQLIN_F32) return run_type<F32>(p, back, s);
    if (dtype == EQLIN_F16) return run_type<F16>(p, back, s);
    return run_type<BF16>(p, back, s);
}

}  // namespace eqlin

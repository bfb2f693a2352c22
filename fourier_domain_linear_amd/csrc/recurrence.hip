// recurrence.hip -- gated linear recurrence over packed sequences, forward and gradients. For every sequence and every
// column (channel and group element), over the tokens in order (reverse: from the last to the first):
//
//   f = sigmoid(forget);  h_t = f_t h_{t-1} + (1 - f_t) x_t;  y_t = h_t, or h_t silu(gate_t)
//
// A stretch of tokens maps the state in front of it to the state behind it by h -> A h + B, A the product of its f; two
// stretches in a row compose to (A' A, A' B + B'). A workgroup takes a chunk of kChunk tokens by a strip of columns: each of
// its waves holds TW tokens in registers (lanes over columns, so every load is one stretch of memory), composes them to
// (A, B), learns through LDS the state in front of its tokens and goes over them again, from the registers, for the results:
// x, forget and gate are read once and y is written once.
//
// The launch takes one of two forms. SEQ: a workgroup goes through a whole sequence, round after round, the next round's tokens on
// their way meanwhile; the fewer sequences there are, the narrower its strips, down to a quarter (a wave's lanes are then 4
// groups that hold stretches of their own), so that more compute units share the work. Where that still leaves too long a way (few
// long sequences), a workgroup a chunk of kChunk tokens: ENDS leaves each chunk's (A, B), CHUNK takes the state in front of its
// chunk through the (A, B) of those before it (JOIN does that between the two for sequences of more than kWindow chunks)
// and does the rest. x and forget are then read twice. (One launch, in which each chunk waits for what those before it publish, was
// built and measured: the hops from chunk to chunk through memory took longer than the second reading, 71 to 89 us against the 61 of then
// for 65536 tokens of 384 columns.)
//
// No atomics, every sum in an order that depends on sizes alone: the same bits every time. Bound by memory where the sequences fill
// the card (bf16, 64 sequences of 196 tokens of 256 x 8 with a gate: 48.5 us, 206 MB, 4.2 TB/s; a large copy reaches 5.0), by a
// round's latency where they do not (16 of 784 tokens of 192 x 4, gate, forward and gradients 63 us, 42 at the copy's rate),
// by the second reading in the split form (one of 65536 tokens of 96 x 4 62 us, 30 at the copy's rate).
//
// Everything is held in fp32; 1 - f is computed as sigmoid(-forget), without the cancellation; results are rounded once.
// Sequences never meet in a sum, so what is not finite in one has no part in another.
#include <type_traits>

#include "stage.h"

namespace eqlin {

namespace {

constexpr int kChunk = kRecurrenceChunk;  // tokens of a chunk and of the distance between marks
constexpr int kWindow = 16;              // chunks whose ends CHUNK goes over by itself
enum Mode { SEQ, ENDS, CHUNK };

// sigmoid(z) and 1 - sigmoid(z), both to a few units of fp32's last place (half types: the hardware's exponential of
// the product with log2 e, relative error up to |z| 2^-24, far below their rounding). FORGET: the reciprocal is corrected once by
// its remainder, since a channel that remembers for hundreds of tokens multiplies as many of them: uncorrected, gradients of
// initial states over up to 4096 tokens were off by 1.25e-6 of their size instead of 3.5e-7 (states 2.0e-7 and 1.0e-7). In the
// half types its exponent is kept below 126, where 1 + e has a reciprocal and e / (1 + e) a value, the minimum passing NaN on; the
// 2^-126 left there are taken off again: a gate of the type's lowest value or of minus infinity has to forget all of a state
// however large, and no f from 2^-101 on changes by it. An output gate is multiplied by its sigmoid, which has to come down to 0
// (gates of the type's lowest value): there the exponential may be infinite, and 1 - sigmoid is the difference, since
// 1 + gate (1 - sigmoid) needs no more.
template <class E, bool FORGET>
__device__ __forceinline__ void sigmoid(float z, float &f, float &rest) {
    float e;
    if constexpr (__is_same(E, F32)) e = expf(-fabsf(z));
    else if constexpr (FORGET) e = __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(-1.4426950408889634f * z, 126.0f));
    else e = __builtin_amdgcn_exp2f(-1.4426950408889634f * z);
    const float d = 1.0f + e;
    float r = __builtin_amdgcn_rcpf(d);
    if constexpr (FORGET) r = fmaf(fmaf(-d, r, 1.0f), r, r);
    if constexpr (__is_same(E, F32)) {
        const float s = e * r;
        f = z >= 0.0f ? r : s;
        rest = z >= 0.0f ? s : r;
    } else {
        f = FORGET ? r - 0x1p-126f : r;
        rest = FORGET ? e * r : 1.0f - r;
    }
}

// ---- sequences ----
//
// Sequence i: its first token, its length, and its first slot: it owns the chunk slots from cu[i] / kChunk + i on, at least
// as many as it has chunks, so the launch needs no lengths on the host. Bounds are forced into the tensors whatever the
// array holds.
struct Seq {
    int t0, len;
    int64_t slot;
};
__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ Seq seq_at(const RecurrenceParams &p, int i) {
    Seq s;
    s.t0 = uniform(clampi(p.cu[i], 0, (int)p.T));
    s.len = uniform(clampi(p.cu[i + 1], s.t0, (int)p.T)) - s.t0;
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
    return uniform(lo);
}

// ---- a wave's tokens ----
//
// A wave is GR groups of 64 / GR lanes; a group takes TW tokens in a row, the next group those after them, a lane EC columns.
// The tokens of a wave from `at` on, in the recurrence's order; those past the end (`past`) and lanes past the last column
// are out of the buffer's range: they load zeros and store nothing. (Zeros have no part in any result: nothing comes after a
// sequence's last token, and nothing comes back from behind it.)
struct Rows {
    int64_t low;  // the lowest row
    int n;        // rows
    bool reverse;
    __device__ __forceinline__ Rows(const RecurrenceParams &p, const Seq &s, int at, int past, int most) : n(min(past - at, most)), reverse(p.reverse) {
        low = reverse ? (int64_t)s.t0 + s.len - at - max(n, 1) : s.t0 + at;
    }
};
// A lane's walk over its tokens of a tensor: 32-bit offsets, rows are at most 2^24 elements apart.
template <class E, int EC, int TW>
struct Cursor {
    typedef typename Elem<E>::T T;
    typedef Pack<E, EC> PK;
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __amdgpu_buffer_rsrc_t rs;
    uint32_t off, step;
    __device__ __forceinline__ Cursor(const Rows &r, const void *t, int64_t stride, int L, int col, int group) {
        const uint32_t row = (uint32_t)stride * (uint32_t)sizeof(T);
        rs = __builtin_amdgcn_make_buffer_rsrc((void *)((const T *)t + r.low * stride), (short)0,
                                               r.n > 0 ? (int)((uint32_t)(r.n - 1) * row + (uint32_t)L * sizeof(T)) : 0, 0x00020000);
        const uint32_t first = r.reverse ? (uint32_t)(r.n - 1 - group * TW) : (uint32_t)(group * TW);
        off = col < L ? first * row + (uint32_t)col * (uint32_t)sizeof(T) : 0xc0000000u;
        step = r.reverse ? 0u - row : row;
    }
    __device__ __forceinline__ void load(PK &v) const {
        if constexpr (PK::kWords == 2) {
            const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
            v.w[0] = u.x, v.w[1] = u.y;
        } else if constexpr (PK::kWords == 1) {
            v.w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
        } else {
            v.w[0] = __builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0);
        }
    }
    __device__ __forceinline__ void store(const float *f) const {
        if constexpr (PK::kWords == 2) {
            const u32x2 u = {__float_as_uint(f[0]), __float_as_uint(f[1])};
            __builtin_amdgcn_raw_buffer_store_b64(u, rs, off, 0, 0);
        } else if constexpr (sizeof(T) == 4) {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[0]), rs, off, 0, 0);
        } else if constexpr (EC == 2) {
            __builtin_amdgcn_raw_buffer_store_b32(pack2<E>(f[0], f[1]), rs, off, 0, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b16(pack1<E>(f[0]), rs, off, 0, 0);
        }
    }
    __device__ __forceinline__ void next() { off += step; }
};
template <class E, int EC, int TW>
__device__ __forceinline__ void load_rows(Pack<E, EC> (&v)[TW], const Rows &r, const void *t, int64_t stride, int L, int col, int group) {
    Cursor<E, EC, TW> c(r, t, stride, L, col, group);
#pragma unroll
    for (int k = 0; k < TW; ++k) {
        c.load(v[k]);
        c.next();
    }
}

// (An idle wave's arrays are cleared: left as they are, the compiler would carry them around the loops in copies.)
template <int N, int EC>
__device__ __forceinline__ void clear(float (&v)[N][EC]) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < EC; ++j) v[k][j] = 0.0f;
}
template <class E, int EC, int N>
__device__ __forceinline__ void clear(Pack<E, EC> (&v)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k].clear();
}

// Over a wave's groups: h -> A h + B of a group's own tokens becomes that of the tokens in front of them (excl), and
// the last group (BACK: the first) gets the whole wave's (A, B). BACK: the order of the groups is the other way round.
template <int GR, int EC, bool BACK>
__device__ __forceinline__ void scan_groups(float *A, float *B, float *xA, float *xB, int group) {
    constexpr int LANES = 64 / GR;
    const int place = BACK ? GR - 1 - group : group;
#pragma unroll
    for (int j = 0; j < EC; ++j) {
#pragma unroll
        for (int m = 1; m < GR; m *= 2) {
            const float a = BACK ? __shfl_down(A[j], m * LANES) : __shfl_up(A[j], m * LANES), b = BACK ? __shfl_down(B[j], m * LANES) : __shfl_up(B[j], m * LANES);
            if (place >= m) B[j] = fmaf(A[j], b, B[j]), A[j] *= a;
        }
        if constexpr (GR > 1) {
            const float a = BACK ? __shfl_down(A[j], LANES) : __shfl_up(A[j], LANES), b = BACK ? __shfl_down(B[j], LANES) : __shfl_up(B[j], LANES);
            xA[j] = place ? a : 1.0f, xB[j] = place ? b : 0.0f;
        } else {
            xA[j] = 1.0f, xB[j] = 0.0f;
        }
    }
}

template <int EC>
__device__ __forceinline__ void load_state(const float *t, int64_t row, int L, int col, float *h) {
    const float *a = t + row * L + col;
    if constexpr (EC == 2) {
        const float2 v = *(const float2 *)a;
        h[0] = v.x, h[1] = v.y;
    } else {
        h[0] = a[0];
    }
}
template <int EC>
__device__ __forceinline__ void store_state(float *t, int64_t row, int L, int col, const float *h) {
    float *a = t + row * L + col;
    if constexpr (EC == 2) *(float2 *)a = make_float2(h[0], h[1]);
    else a[0] = h[0];
}

// ---- the states in front of chunks ----
//
// The (A, B) of the chunk in `slot`, columns col .. col + EC.
template <int EC>
__device__ __forceinline__ void store_end(float2 *ends, int64_t slot, int L, int col, const float *a, const float *b) {
#pragma unroll
    for (int j = 0; j < EC; ++j) ends[slot * L + col + j] = make_float2(a[j], b[j]);
}

// h through the ends of the n chunks in front of a chunk (slot0 + dir c is the slot of the c-th): every wave fetches its
// share of the first kWindow, on its way while tokens are worked on; EC waves take 64 columns each through them and tell
// the others. (More than kWindow are there only where `longest` said too little.)
template <int EC>
struct Window {
    float2 ends[kWindow][64 * EC];
    float state[64 * EC];
};
template <int EC, int W>
struct Fold {
    static constexpr int SHARE = (kWindow + W - 1) / W;
    const float2 *ends;  // of the lane's columns of chunk 0
    int64_t step;
    int n, lane, wave;
    float2 v[SHARE][EC];
    __device__ __forceinline__ Fold(const float2 *all, int64_t slot0, int dir, int count, int L, int col, int ln, int wv)
        : ends(all + slot0 * L + col), step((int64_t)dir * L), n(count), lane(ln), wave(wv) {
        fetch(0);
    }
    __device__ __forceinline__ void fetch(int at) {
#pragma unroll
        for (int q = 0; q < SHARE; ++q)
            if (at + wave + q * W < n)
#pragma unroll
                for (int j = 0; j < EC; ++j) v[q][j] = ends[(at + wave + q * W) * step + j];
    }
    __device__ __forceinline__ void finish(Window<EC> &lds, float *h) {
        if (wave == 0)
#pragma unroll
            for (int j = 0; j < EC; ++j) lds.state[lane * EC + j] = h[j];
        for (int at = 0;;) {
#pragma unroll
            for (int q = 0; q < SHARE; ++q)
                if (wave + q * W < min(kWindow, n - at))
#pragma unroll
                    for (int j = 0; j < EC; ++j) lds.ends[wave + q * W][lane * EC + j] = v[q][j];
            __syncthreads();
            if (n == 0) break;
            if (wave < EC) {
                float b = lds.state[wave * 64 + lane];
                const int m = min(kWindow, n - at);
#pragma unroll 4
                for (int c = 0; c < m; ++c) {
                    const float2 e = lds.ends[c][wave * 64 + lane];
                    b = fmaf(e.x, b, e.y);
                }
                lds.state[wave * 64 + lane] = b;
            }
            __syncthreads();
            if ((at += kWindow) >= n) break;
            fetch(at);
        }
#pragma unroll
        for (int j = 0; j < EC; ++j) h[j] = lds.state[lane * EC + j];
    }
};

// JOIN, for sequences of any length: the states in front of all chunks of a sequence but the first (BACK: what comes back
// from behind all but the last). 16 columns a workgroup; its groups of 16 lanes compose kShare chunks each, learn through LDS the
// state in front of them, and go over them again from the registers.
constexpr int kShare = 16;
template <bool BACK, int GROUPS>
__global__ void __launch_bounds__(16 * GROUPS) k_recurrence_join(const RecurrenceParams p, int strips, int64_t units) {
    __shared__ float2 parts[2][GROUPS][16];
    const int L = p.C << p.lg, c16 = threadIdx.x & 15, group = threadIdx.x >> 4;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int i = (int)(unit / strips), u = (int)(unit - (int64_t)i * strips) * 16 + c16, col = u < L ? u : 0;
        const Seq s = seq_at(p, i);
        const int n = (s.len + kChunk - 1) / kChunk - 1;  // ends to go through
        float h = 0.0f;                                   // (the first end on the way is a state: initial states and dfinal are in it)
        auto slot = [&](int c) { return s.slot + (BACK ? n - c : c); };  // of the c-th chunk on the way
        for (int at = 0, buf = 0; at < n; at += GROUPS * kShare, buf ^= 1) {
            const int c0 = at + group * kShare;
            float2 e[kShare];
#pragma unroll
            for (int k = 0; k < kShare; ++k) e[k] = c0 + k < n ? p.ends[slot(c0 + k) * L + col] : make_float2(1.0f, 0.0f);
            float A = 1.0f, B = 0.0f;  // (past the last end: nothing changes)
#pragma unroll
            for (int k = 0; k < kShare; ++k) A *= e[k].x, B = fmaf(e[k].x, B, e[k].y);
            parts[buf][group][c16] = make_float2(A, B);
            __syncthreads();
            float mine = h;
            const int groups = min(GROUPS, (n - at + kShare - 1) / kShare);
#pragma unroll 4
            for (int g = 0; g < groups; ++g) {
                const float2 q = parts[buf][g][c16];
                if (g == group) mine = h;
                h = fmaf(q.x, h, q.y);
            }
#pragma unroll
            for (int k = 0; k < kShare; ++k) {
                mine = fmaf(e[k].x, mine, e[k].y);
                if (c0 + k < n && u < L) p.carry[slot(c0 + k + 1) * L + col] = mine;
            }
        }
        __syncthreads();  // the parts are used again
    }
}

// What a workgroup works on: a strip of columns of a sequence (SEQ), or of one chunk of it.
struct Unit {
    Seq s;
    int i, tile, last, col;  // tile: the first chunk; last: the sequence's last; col: the lane's first column
    bool none;               // a slot without a chunk
};
// kXcds neighbouring workgroups are on as many XCDs: CHUNK goes through the units from the last group of them to the first.
constexpr int kXcds = 8;
template <Mode MODE, int EC, int GR>
__device__ __forceinline__ Unit unit_at(const RecurrenceParams &p, int64_t unit, int strips, int64_t units) {
    Unit u;
    if (MODE == CHUNK) unit = (units - 1) / kXcds * kXcds - unit / kXcds * kXcds + unit % kXcds;
    const int64_t id = unit / strips;
    u.none = unit >= units;
    u.col = ((int)(unit - id * strips) * (64 / GR) + (threadIdx.x & (64 / GR - 1))) * EC;
    u.i = MODE == SEQ ? (int)id : seq_of_slot(p, id);
    u.s = seq_at(p, u.i);
    u.last = (u.s.len + kChunk - 1) / kChunk - 1;
    u.tile = MODE == SEQ ? 0 : uniform((int)(id - u.s.slot));
    u.none = u.none || (MODE != SEQ && (u.tile < 0 || u.tile > u.last));
    return u;
}

template <Mode MODE>
__device__ __forceinline__ int64_t padded(int64_t units) { return MODE == CHUNK ? (units + kXcds - 1) / kXcds * kXcds : units; }

// States of sequences without tokens, which have no chunk: final = state (dstate = dfinal).
__device__ __forceinline__ void empty_sequences(const RecurrenceParams &p, const float *from, float *to) {
    if (!to || to == from) return;
    const int L = p.C << p.lg;
    for (int i = blockIdx.x; i < p.B; i += gridDim.x)
        if (seq_at(p, i).len == 0)
            for (int e = threadIdx.x; e < L; e += blockDim.x) to[(int64_t)i * L + e] = from ? from[(int64_t)i * L + e] : 0.0f;
}

// LDS of the kernels: what the waves of a workgroup tell each other, in SEQ twice, so that one barrier a round is enough.
template <int EC, int W, int N, int GR, Mode MODE>
struct Shared {
    float ends[MODE == SEQ ? 2 : 1][N][W][64 / GR * EC];
    float start[2][64 / GR * EC];
    std::conditional_t<MODE == CHUNK, Window<EC>, char> window;
};

template <class E, int EC, int TW, int W, int GR, bool GATE, Mode MODE>
__global__ void __launch_bounds__(64 * W) k_recurrence(const RecurrenceParams p, int strips, int64_t units) {
    typedef Pack<E, EC> PK;
    constexpr int LANES = 64 / GR, SPAN = TW * GR, ROUND = SPAN * W;
    static_assert(MODE == SEQ ? (kChunk % ROUND == 0 || (ROUND % kChunk == 0 && kChunk % TW == 0)) : ROUND == kChunk && GR == 1, "marks lie between groups");
    __shared__ Shared<EC, W, 2, GR, MODE> lds;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), group = lane / LANES, own = lane % LANES * EC, L = p.C << p.lg;
    int buf = 0;
    if constexpr (MODE == ENDS) empty_sequences(p, p.state, p.final);
    for (int64_t unit = blockIdx.x; unit < padded<MODE>(units); unit += gridDim.x) {
        const Unit u = unit_at<MODE, EC, GR>(p, unit, strips, units);
        if (u.none || (MODE == ENDS && u.tile == u.last)) continue;  // (nobody asks for a last chunk's end)
        const bool in = u.col < L;
        const int col = in ? u.col : 0;
        // The initial state is read by wave 0 alone, which hands it on through LDS before anything is written; a final one is
        // written by who has the last token. The two may be one buffer, so of a sequence of several chunks ENDS alone reads
        // the state: it leaves it in the last chunk's place, and the state behind the first chunk as that chunk's end.
        float carry[EC];
#pragma unroll
        for (int j = 0; j < EC; ++j) carry[j] = 0.0f;
        if (wave == 0 && p.state && u.tile == 0 && (MODE != CHUNK || u.last == 0)) load_state<EC>(p.state, u.i, L, col, carry);
        Fold<EC, W> fold(p.ends, u.s.slot, 1, MODE == CHUNK && !p.carry ? u.tile : 0, L, col, lane, wave);
        if constexpr (MODE == CHUNK) {
            if (u.tile == 0 && u.last > 0)
#pragma unroll
                for (int j = 0; j < EC; ++j) carry[j] = p.ends[(u.s.slot + u.last) * L + col + j].y;
            if (u.tile > 0 && p.carry) load_state<EC>(p.carry, u.s.slot + u.tile, L, col, carry);
        }
        if (u.s.len == 0) {
            if (wave == 0 && group == 0 && in && p.final) store_state<EC>(p.final, u.i, L, col, carry);
            continue;
        }
        const int stop = MODE == SEQ ? u.s.len : min(u.s.len, (u.tile + 1) * kChunk);
        PK x[TW], z[TW], o[GATE ? TW : 1];
        auto fetch = [&](int at) {  // a round's tokens; in SEQ they are on their way while the round before is finished
            const Rows r(p, u.s, at + wave * SPAN, min(stop, at + ROUND), SPAN);
            if (r.n <= 0) return;
            load_rows(z, r, p.f, p.ft, L, u.col, group);
            load_rows(x, r, p.x, p.xt, L, u.col, group);
            if constexpr (GATE) load_rows(o, r, p.o, p.ot, L, u.col, group);
        };
        clear(x), clear(z), clear(o);
        fetch(u.tile * kChunk);
        for (int at = u.tile * kChunk; at < stop; at += ROUND, buf ^= MODE == SEQ) {
            const int t = at + wave * SPAN, past = min(stop, at + ROUND);
            float f[TW][EC], b[TW][EC], s[GATE ? TW : 1][EC];  // s: silu(gate)
            float A[EC], B[EC], xA[EC], xB[EC];
#pragma unroll
            for (int j = 0; j < EC; ++j) A[j] = 1.0f, B[j] = 0.0f;
            if (t < past) {
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    float v[EC], w[EC], g[EC];
                    x[k].unpack(v);
                    z[k].unpack(w);
                    if constexpr (GATE) o[k].unpack(g);
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        float rest;
                        sigmoid<E, true>(w[j], f[k][j], rest);
                        b[k][j] = rest * v[j];
                        A[j] *= f[k][j];
                        B[j] = fmaf(f[k][j], B[j], b[k][j]);
                        if constexpr (GATE) {
                            sigmoid<E, false>(g[j], s[k][j], rest);
                            s[k][j] *= g[j];
                        }
                    }
                }
            } else {
                clear(f), clear(b), clear(s);
            }
            if (MODE == SEQ && at + ROUND < stop) fetch(at + ROUND);
            scan_groups<GR, EC, false>(A, B, xA, xB, group);
            if (group == GR - 1)
#pragma unroll
                for (int j = 0; j < EC; ++j) lds.ends[buf][0][wave][own + j] = A[j], lds.ends[buf][1][wave][own + j] = B[j];
            if (MODE == SEQ && wave == 0 && group == 0)
#pragma unroll
                for (int j = 0; j < EC; ++j) lds.start[buf][own + j] = carry[j];
            if constexpr (MODE == CHUNK) fold.finish(lds.window, carry);
            else __syncthreads();
            float h[EC];
            if constexpr (MODE == ENDS) {
                float total[EC], sum[EC];  // (A, B) of the chunk
#pragma unroll
                for (int j = 0; j < EC; ++j) total[j] = 1.0f, sum[j] = 0.0f;
#pragma unroll 2
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        const float aw = lds.ends[buf][0][w][own + j];
                        total[j] *= aw;
                        sum[j] = fmaf(aw, sum[j], lds.ends[buf][1][w][own + j]);
                    }
                if (wave == 0 && in) {
                    if (u.tile == 0) {
                        const float zero[EC] = {};
                        store_end<EC>(p.ends, u.s.slot + u.last, L, col, zero, carry);
#pragma unroll
                        for (int j = 0; j < EC; ++j) sum[j] = fmaf(total[j], carry[j], sum[j]), total[j] = 0.0f;
                    }
                    store_end<EC>(p.ends, u.s.slot + u.tile, L, col, total, sum);
                }
            } else {
                if constexpr (MODE == SEQ)
#pragma unroll
                    for (int j = 0; j < EC; ++j) carry[j] = lds.start[buf][own + j];
#pragma unroll
                for (int j = 0; j < EC; ++j) h[j] = carry[j];
#pragma unroll 2
                for (int w = 0; w < (MODE == SEQ ? W : wave); ++w) {
                    if (MODE == SEQ && w == wave)
#pragma unroll
                        for (int j = 0; j < EC; ++j) h[j] = carry[j];
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        float &c = MODE == SEQ ? carry[j] : h[j];
                        c = fmaf(lds.ends[buf][0][w][own + j], c, lds.ends[buf][1][w][own + j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < EC; ++j)
                    if (GR > 1) h[j] = fmaf(xA[j], h[j], xB[j]);
                const int mine = t + group * TW;  // the group's first token
                if (p.marks && in && mine < past && mine % kChunk == 0) store_state<EC>(p.marks, u.s.slot + mine / kChunk, L, col, h);
                if (p.final && in && past == u.s.len && mine < past && mine + TW >= past) {  // the last token's group
                    float last[EC];
#pragma unroll
                    for (int j = 0; j < EC; ++j) last[j] = h[j];
#pragma unroll
                    for (int k = 0; k < TW; ++k)
                        if (mine + k < past)
#pragma unroll
                            for (int j = 0; j < EC; ++j) last[j] = fmaf(f[k][j], last[j], b[k][j]);
                    store_state<EC>(p.final, u.i, L, col, last);
                }
                const Rows r(p, u.s, t, past, SPAN);
                if (r.n > 0) {
                    Cursor<E, EC, TW> out(r, p.y, p.yt, L, u.col, group);
#pragma unroll
                    for (int k = 0; k < TW; ++k) {
                        float y[EC];
#pragma unroll
                        for (int j = 0; j < EC; ++j) {
                            y[j] = h[j] = fmaf(f[k][j], h[j], b[k][j]);
                            if constexpr (GATE) y[j] *= s[k][j];
                        }
                        out.store(y);
                        out.next();
                    }
                }
            }
        }
        if (MODE != SEQ) __syncthreads();  // the exchange is used again
    }
}

// ---- gradients ----
//
//   dh_t = dy_t silu(gate_t) + f_{t+1} dh_{t+1} (+ dfinal at the last token)
//   dx = (1 - f) dh;  dforget = dh (h_{t-1} - x) f (1 - f);  dgate = dy h silu'(gate);  dstate = f_1 dh_1
//
// What goes back over a stretch's start, g_t = f_t dh_t, is composed from the last token on with the same A:
// g -> A g + B'. The states come again from x and forget, exactly as the forward had them, from its marks: the states in
// front of each chunk. SEQ, ENDS and CHUNK as above, the chunks taken from the last to the first.
template <class E, int EC, int TW, int W, int GR, bool GATE, Mode MODE>
__global__ void __launch_bounds__(64 * W) k_recurrence_bwd(const RecurrenceParams p, int strips, int64_t units) {
    typedef Pack<E, EC> PK;
    constexpr int LANES = 64 / GR, SPAN = TW * GR, ROUND = SPAN * W;
    constexpr int WC = kChunk / SPAN;  // waves of a chunk
    static_assert(kChunk % SPAN == 0 && (MODE == SEQ ? ROUND % kChunk == 0 : ROUND == kChunk && GR == 1), "a chunk is whole waves");
    __shared__ Shared<EC, W, 3, GR, MODE> lds;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), group = lane / LANES, own = lane % LANES * EC, L = p.C << p.lg;
    int buf = 0;
    if constexpr (MODE == ENDS) empty_sequences(p, p.dfinal, p.dstate);
    for (int64_t unit = blockIdx.x; unit < padded<MODE>(units); unit += gridDim.x) {
        const Unit u = unit_at<MODE, EC, GR>(p, unit, strips, units);
        if (u.none || (MODE == ENDS && u.tile == 0)) continue;  // (nobody asks what leaves the first chunk)
        const bool in = u.col < L;
        const int col = in ? u.col : 0;
        float g[EC], end[EC];  // what comes back from behind the round (nothing, behind the last); dfinal
#pragma unroll
        for (int j = 0; j < EC; ++j) g[j] = end[j] = 0.0f;
        if (p.dfinal) load_state<EC>(p.dfinal, u.i, L, col, end);
        if (u.s.len == 0) {
            if (wave == 0 && group == 0 && in && p.dstate) store_state<EC>(p.dstate, u.i, L, col, end);
            continue;
        }
        Fold<EC, W> fold(p.ends, u.s.slot + u.last, -1, MODE == CHUNK && !p.carry ? u.last - u.tile : 0, L, col, lane, wave);
        if (MODE == CHUNK && p.carry && u.tile < u.last) load_state<EC>(p.carry, u.s.slot + u.tile, L, col, g);
        const int first = MODE == SEQ ? 0 : u.tile * kChunk;
        for (int at = MODE == SEQ ? (u.s.len - 1) / ROUND * ROUND : first; at >= first; at -= ROUND, buf ^= MODE == SEQ) {
            const int t = at + wave * SPAN, past = min(u.s.len, at + ROUND), mine = t + group * TW;
            const Rows r(p, u.s, t, past, SPAN);
            PK x[TW];
            // d: dy silu(gate), then dh; q: dy silu'(gate)
            float f[TW][EC], rest[TW][EC], d[TW][EC], q[GATE ? TW : 1][EC];
            float A[EC], B[EC], R[EC], bA[EC], xA[EC], xB[EC], yA[EC], yR[EC], h[EC];
#pragma unroll
            for (int j = 0; j < EC; ++j) A[j] = 1.0f, B[j] = R[j] = h[j] = 0.0f;
            if (MODE != ENDS && r.n > 0) load_state<EC>(p.marks, u.s.slot + t / kChunk, L, col, h);
            if (r.n > 0) {
                PK z[TW], dy[TW], o[GATE ? TW : 1];
                load_rows(z, r, p.f, p.ft, L, u.col, group);
                load_rows(dy, r, p.dy, p.dyt, L, u.col, group);
                if constexpr (GATE) load_rows(o, r, p.o, p.ot, L, u.col, group);
                if constexpr (MODE != ENDS) load_rows(x, r, p.x, p.xt, L, u.col, group);
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    float v[EC], w[EC], s[EC];
                    z[k].unpack(w);
                    dy[k].unpack(d[k]);
                    if constexpr (MODE != ENDS) x[k].unpack(v);
                    if constexpr (GATE) o[k].unpack(s);
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        sigmoid<E, true>(w[j], f[k][j], rest[k][j]);
                        if constexpr (GATE) {
                            float sig, other;
                            sigmoid<E, false>(s[j], sig, other);
                            const float t = d[k][j] * sig;
                            q[k][j] = t * fmaf(s[j], other, 1.0f);
                            d[k][j] = t * s[j];
                        }
                        A[j] *= f[k][j];
                        if constexpr (MODE != ENDS) B[j] = fmaf(f[k][j], B[j], rest[k][j] * v[j]);
                    }
                }
                if (p.dfinal && past == u.s.len && mine < past && mine + TW >= past)  // the last token's group
#pragma unroll
                    for (int k = 0; k < TW; ++k)
                        if (mine + k + 1 == past)
#pragma unroll
                            for (int j = 0; j < EC; ++j) d[k][j] += end[j];
#pragma unroll
                for (int k = TW - 1; k >= 0; --k)
#pragma unroll
                    for (int j = 0; j < EC; ++j) R[j] = f[k][j] * (d[k][j] + R[j]);
            } else {
                clear(f), clear(rest), clear(d), clear(q), clear(x);
            }
            // the groups' A B forwards (a chunk's states), A R backwards
#pragma unroll
            for (int j = 0; j < EC; ++j) bA[j] = A[j];
            if constexpr (MODE != ENDS) scan_groups<GR, EC, false>(A, B, xA, xB, group);
            scan_groups<GR, EC, true>(bA, R, yA, yR, group);
            if (group == GR - 1)
#pragma unroll
                for (int j = 0; j < EC; ++j) lds.ends[buf][0][wave][own + j] = A[j], lds.ends[buf][1][wave][own + j] = B[j];
            if (group == 0)
#pragma unroll
                for (int j = 0; j < EC; ++j) lds.ends[buf][2][wave][own + j] = R[j];
            if constexpr (MODE == CHUNK) fold.finish(lds.window, g);
            else __syncthreads();
            if constexpr (MODE != ENDS) {
#pragma unroll 2
                for (int w = wave / WC * WC; w < wave; ++w)
#pragma unroll
                    for (int j = 0; j < EC; ++j) h[j] = fmaf(lds.ends[buf][0][w][own + j], h[j], lds.ends[buf][1][w][own + j]);
#pragma unroll
                for (int j = 0; j < EC; ++j)
                    if (GR > 1) h[j] = fmaf(xA[j], h[j], xB[j]);
            }
            float total[EC], back[EC];
#pragma unroll
            for (int j = 0; j < EC; ++j) total[j] = 1.0f, back[j] = g[j];
#pragma unroll 2
            for (int w = W - 1; w >= 0; --w) {
                if (w == wave)
#pragma unroll
                    for (int j = 0; j < EC; ++j) back[j] = g[j];
#pragma unroll
                for (int j = 0; j < EC; ++j) {
                    const float aw = lds.ends[buf][0][w][own + j];
                    if (MODE == ENDS) total[j] *= aw;
                    g[j] = fmaf(aw, g[j], lds.ends[buf][2][w][own + j]);
                }
            }
            if constexpr (MODE == ENDS) {
                if (wave == 0 && in) store_end<EC>(p.ends, u.s.slot + u.tile, L, col, total, g);
            } else if (r.n > 0) {
#pragma unroll
                for (int j = 0; j < EC; ++j)
                    if (GR > 1) back[j] = fmaf(yA[j], back[j], yR[j]);
#pragma unroll
                for (int k = TW - 1; k >= 0; --k)
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        d[k][j] += back[j];
                        back[j] = f[k][j] * d[k][j];
                    }
                Cursor<E, EC, TW> ox(r, p.dx, p.dxt, L, u.col, group), of(r, p.df, p.dft, L, u.col, group), og(r, p.dgo, p.dgot, L, u.col, group);
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    float v[EC], w[EC], s[EC];
                    x[k].unpack(v);
#pragma unroll
                    for (int j = 0; j < EC; ++j) {
                        const float gx = rest[k][j] * d[k][j];
                        // f first and h and x apart: dh (h - x) and h - x may be beyond fp32 where the gradient is not, or is 0
                        const float t = gx * f[k][j];
                        w[j] = fmaf(t, h[j], -(t * v[j]));
                        h[j] = fmaf(f[k][j], h[j], rest[k][j] * v[j]);
                        if constexpr (GATE) s[j] = q[k][j] * h[j];
                        v[j] = gx;
                    }
                    ox.store(v);
                    of.store(w);
                    if constexpr (GATE)
                        if (p.dgo) og.store(s);
                    ox.next(), of.next(), og.next();
                }
            }
        }
        if (MODE != ENDS && (MODE == SEQ || u.tile == 0) && wave == 0 && group == 0 && in && p.dstate) store_state<EC>(p.dstate, u.i, L, col, g);
        if (MODE != SEQ) __syncthreads();  // the exchange is used again
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
    auto strips_of = [&](int columns) { return (int)((L + columns - 1) / columns); };
    auto grid = [](int64_t n) { return dim3((unsigned)std::min<int64_t>((n + kXcds - 1) / kXcds * kXcds, kGrid)); };
    int strips;
    int64_t units;
#define EQLIN_RECURRENCE(K, TW, W, GR, GATED, MODE)              \
    strips = strips_of(64 / GR * EC);                            \
    units = (MODE == SEQ ? (int64_t)p.B : p.slots) * strips;     \
    hipLaunchKernelGGL((K<E, EC, TW, W, GR, GATED, MODE>), grid(units), dim3(64 * W), 0, s, p, strips, units)
    // JOIN: 16 groups take up to 256 chunks at once (24 sequences of up to 49: 4 us, 64 groups 14 us), 64 groups 1024
#define EQLIN_JOIN(BACK)                                                                                                              \
    do {                                                                                                                              \
        strips = strips_of(16);                                                                                                       \
        units = (int64_t)p.B * strips;                                                                                                \
        if (p.longest <= 256 * kChunk) hipLaunchKernelGGL((k_recurrence_join<BACK, 16>), grid(units), dim3(256), 0, s, p, strips, units); \
        else hipLaunchKernelGGL((k_recurrence_join<BACK, 64>), grid(units), dim3(1024), 0, s, p, strips, units);                      \
    } while (0)
    if (!p.split) {
        if (back) {
            if (p.groups == 4) { EQLIN_RECURRENCE(k_recurrence_bwd, 8, 8, 4, GATE, SEQ); }
            else if (p.groups == 2) { EQLIN_RECURRENCE(k_recurrence_bwd, 8, 8, 2, GATE, SEQ); }
            else { EQLIN_RECURRENCE(k_recurrence_bwd, 8, 8, 1, GATE, SEQ); }
        } else if (p.longest <= 1) {
            EQLIN_RECURRENCE(k_recurrence, 1, 1, 1, GATE, SEQ);
        } else if (p.longest <= 8) {
            EQLIN_RECURRENCE(k_recurrence, 8, 1, 1, GATE, SEQ);
        } else {
            if (p.groups == 4) { EQLIN_RECURRENCE(k_recurrence, 8, 8, 4, GATE, SEQ); }
            else if (p.groups == 2) { EQLIN_RECURRENCE(k_recurrence, 8, 8, 2, GATE, SEQ); }
            else { EQLIN_RECURRENCE(k_recurrence, 8, 8, 1, GATE, SEQ); }
        }
    } else if (back) {
        EQLIN_RECURRENCE(k_recurrence_bwd, 8, 8, 1, GATE, ENDS);
        if (p.carry) EQLIN_JOIN(true);
        EQLIN_RECURRENCE(k_recurrence_bwd, 8, 8, 1, GATE, CHUNK);
    } else {
        EQLIN_RECURRENCE(k_recurrence, 8, 8, 1, false, ENDS);
        if (p.carry) EQLIN_JOIN(false);
        EQLIN_RECURRENCE(k_recurrence, 8, 8, 1, GATE, CHUNK);
    }
#undef EQLIN_RECURRENCE
#undef EQLIN_JOIN
    return hipGetLastError();
}

template <class E>
hipError_t run_type(const RecurrenceParams &p, bool back, hipStream_t s) {
    if (in_pairs<E>(p, back)) return p.o ? run<E, 2, true>(p, back, s) : run<E, 2, false>(p, back, s);
    return p.o ? run<E, 1, true>(p, back, s) : run<E, 1, false>(p, back, s);
}

}  // namespace

// The form of a launch, by its time in us on an MI355X as measured over widths of 256 to 2048 columns, 1 to 128 sequences of
// 64 to 4096 tokens. floor: the bytes that must move, at 5 TB/s. SEQ takes `round` for each 64 tokens a group of lanes of the longest
// sequence, and a part of the floor beside it; narrower strips (more groups) take longer rounds and more of the memory's time (a row's
// stretch is 64 bytes of a half type with 4), but more workgroups and fewer rounds. The split form reads twice.
// Measured in us, 1, 2, 4 groups, split (the form that is taken in brackets; over 64 such points it is within 6 % of the best):
//                    32 sequences of 1024 x 256    128 of 1024 x 256          2 of 4096 x 256            64 of 196 x 2048
//   bf16             34.4 21.4 [16.9] 24.9        41.6 [42.2] 58.3 82.6      120.7 67.5 35.6 [15.8]    [33.1] 36.6 54.5 68.0
//   bf16 gate        42.1 24.5 [21.5] 27.8        [52.5] 54.9 76.6 94.3      155.9 85.1 45.6 [17.5]    [45.2] 46.9 67.8 80.6
//   bf16 back        48.2 30.2 [27.3] 28.3        [75.2] 70.3 99.7 103.8     174.4 96.5 54.1 [17.0]    [51.1] 57.0 91.9 85.4
//   bf16 gate back   62.0 38.1 [36.0] 42.5        [102.6] 107.6 149.1 159.6  233.8 127.9 70.0 [19.2]   [91.9] 88.3 125.6 132.5
//   fp32             46.2 29.6 [21.9] 36.3        [84.6] 81.4 88.4 134.4     161.7 86.8 45.6 [20.2]    [60.3] 61.8 67.9 111.3
//   fp32 gate        74.5 45.2 [31.5] 44.3        [113.9] 112.5 123.4 155.0  246.8 128.1 66.5 [23.1]   [87.0] 99.1 115.1 131.6
//   fp32 back        88.4 49.8 [36.5] 47.9        [140.8] 135.2 148.6 174.9  283.5 133.4 71.7 [23.8]   [107.2] 105.2 109.8 133.7
//   fp32 gate back   128.8 72.4 [52.6] 72.8       [193.9] 195.9 211.5 282.3  419.8 202.3 106.1 [27.0]  [163.3] 160.7 169.5 224.6
// The number of sequences has no part in it, and JOIN takes a workgroup a sequence and 16 columns whatever the sequence's length: a long
// prompt beside many single tokens pays for them (bf16, one of 32768 tokens of 384 columns: 36 us alone, 43 beside 100 single
// tokens, 75 beside 512, 112 beside 1000, which take 3.4 in a call of their own).
void plan_recurrence(RecurrenceParams &p, eqlin_dtype_t dtype, bool back) {
    const int64_t L = (int64_t)p.C << p.lg;
    const bool f32 = dtype == EQLIN_F32;
    const int gate = p.o ? 1 : 0;
    p.slots = p.T / kChunk + p.B;
    p.joined = (p.longest + kChunk - 1) / kChunk > kWindow + 1;
    const double floor = (double)p.T * L * (f32 ? 4 : 2) * (back ? 5 + 2 * gate : 3 + gate) / 5e6;
    const double round = (f32 ? (back ? 4.0 + 1.3 * gate : 2.5 + 0.8 * gate) : (back ? 2.6 + 0.95 * gate : 1.77 + 0.58 * gate)) * (L % 2 ? 0.6 : 1.0);
    const struct {
        int groups;
        double round, beside, least;  // a round's time, the share of the floor beside it, the least share
    } forms[] = {{1, 1.0, 0.3, 1.0}, {2, 1.1, back ? 0.35 : 0.2, back && gate ? 1.15 : 1.05}, {4, 1.22, back ? 0.7 : 0.45, f32 ? 1.1 : 1.6}};
    double best = (p.joined ? 12.0 : 8.0) + (back ? 1.3 + 0.2 * gate : 1.6 - 0.1 * gate) * floor;
    p.split = p.longest > kChunk;
    p.groups = 1;
    for (const auto &f : forms) {
        const int64_t span = (int64_t)kChunk * f.groups;
        const double t = std::max(f.least * floor, 2.0 + (double)((p.longest + span - 1) / span) * f.round * round + f.beside * floor);
        if (p.longest > kChunk && t < best) best = t, p.split = false, p.groups = f.groups;
    }
}

// The chunks' ends, and the states in front of them where JOIN runs.
size_t recurrence_workspace_bytes(const RecurrenceParams &p) {
    const size_t states = (size_t)p.slots * ((size_t)p.C << p.lg);
    return !p.split ? 0 : states * (sizeof(float2) + (p.joined ? sizeof(float) : 0));
}

hipError_t launch_recurrence(RecurrenceParams p, eqlin_dtype_t dtype, bool back, void *ws, hipStream_t s) {
    if (p.split) {
        p.ends = (float2 *)ws;
        p.carry = p.joined ? (float *)(p.ends + p.slots * ((int64_t)p.C << p.lg)) : nullptr;
    }
    if (dtype == EQLIN_F32) return run_type<F32>(p, back, s);
    if (dtype == EQLIN_F16) return run_type<F16>(p, back, s);
    return run_type<BF16>(p, back, s);
}

}  // namespace eqlin

// rotary.hip -- rotary positions over one to four axes. Pair j (channels j and j + P of a head) belongs to
// one axis and turns by freq[j] times the token's position on it. The last two axes are (row, column), and
// group element g sees them turned by g^-1 (p_g = R^-g p; D4: S^b R^-a p), R(row, col) = (-col, row) the
// quarter turn: turning the image and shifting the group axis by one then commutes with the rotation.
//
// The angle is taken in turns in fp64 (position x frequency, less its whole turns), so that a position in
// the millions is as exact as a small one, and its sine and cosine in fp32 (half types: the hardware's,
// absolute error about 1e-6, far below a half's rounding; fp32: the library's). They are computed once a
// lane and used for every head that it takes.
//
// Bound by memory: x read once, y written once, in 16-byte vectors. bf16, 12544 tokens, 32 heads of 16 x 8: 33 to 38 us
// (206 MB, 5.4 to 6.3 TB/s, part of it in the last cache; a large copy reaches 5.1). Off 16 bytes the pairs are moved one by
// one: 154 us.
#include "stage.h"

namespace eqlin {

namespace {

// sine and cosine of t turns
template <class E>
__device__ __forceinline__ void turn(double t, float &c, float &s) {
    const float f = (float)(t - rint(t));
    if constexpr (__is_same(E, F32)) {
        sincospif(2.0f * f, &s, &c);
    } else {
        s = __builtin_amdgcn_sinf(f);
        c = __builtin_amdgcn_cosf(f);
    }
}

// cos and sin of pair j's angle for the group elements g0 .. g0 + N - 1 (N a power of two, g0 a multiple of it). Seen
// from g, a row (or column) position r is A cos(2 pi g / G) + B sin(2 pi g / G) with A the position itself and B the other
// axis's, signed; half a turn on, the angle is the negative one, so G = 8 takes four sines and cosines a channel and
// D4 two.
template <class E, int LG, int N>
__device__ __forceinline__ void rotary_angles(const RotaryParams &p, const int *pos, int j, int g0, float *c, float *s) {
    constexpr int G = 1 << LG;
    int axis = 0;
    while (axis + 1 < p.axes && j >= p.end[axis]) ++axis;
    const int back = p.axes - axis;  // 2: rows, 1: columns
    const double f = p.inverse ? -p.freq[j] : p.freq[j];
    if (LG == 0 || p.axes == 1 || back > 2) {  // the same for every g
        float c1, s1;
        turn<E>(pos[axis] * f, c1, s1);
#pragma unroll
        for (int k = 0; k < N; ++k) c[k] = c1, s[k] = s1;
        return;
    }
    const double row = pos[p.axes - 2] * f, col = pos[p.axes - 1] * f;
    const double A = back == 2 ? row : col, B = back == 2 ? col : -row;
    if constexpr (LG == 3) {
        if (p.d4) {  // a + 4 b: quarter turns a; the mirror b turns the columns' sign
            float ca, sa, cb, sb;
            turn<E>(A, ca, sa);
            turn<E>(B, cb, sb);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int g = g0 + k;
                const float x = (g & 1) ? sb : sa, y = (g & 2) ? -x : x;
                c[k] = (g & 1) ? cb : ca;
                s[k] = (g & 4) && back == 1 ? -y : y;
            }
            return;
        }
    }
    constexpr int H = G > 1 ? G / 2 : 1;  // distinct up to sign
    float ch[H], sh[H];
    turn<E>(A, ch[0], sh[0]);
    if constexpr (H >= 2) turn<E>(B, ch[H / 2], sh[H / 2]);
    if constexpr (H == 4) {
        const double h = 0.70710678118654752440;
        turn<E>((A + B) * h, ch[1], sh[1]);
        turn<E>((B - A) * h, ch[3], sh[3]);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {  // (N < G only where the vector is half a channel: g0 is 0 or G / 2)
        const bool neg = ((g0 + k) & H) != 0 && G > 1;
        c[k] = ch[k % H];
        s[k] = neg ? -sh[k % H] : sh[k % H];
    }
}

// Vectors: lanes run over the vectors of a head's first half, then over heads; HL heads at a time a token.
template <class E, int LG>
__global__ void __launch_bounds__(256) k_rotary(const RotaryParams p, int nv, int nr, int HL) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    constexpr int V = EL::V, G = 1 << LG, N = G < V ? G : V;  // group elements of one channel in a vector
    const int lanes = (nv + nr) * HL;                         // lanes a token; nr vectors past the pairs are copied
    const int PG = p.P << LG;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < p.N * lanes; id += (int64_t)gridDim.x * 256) {
        const int64_t n = id / lanes;
        const int sub = (int)(id - n * lanes), h0 = sub / (nv + nr), v = sub % (nv + nr);
        const T *x = (const T *)p.x + n * p.xt;
        T *y = (T *)p.y + n * p.yt;
        if (v >= nv) {
            const int e = 2 * PG + (v - nv) * V;
            for (int h = h0; h < p.H; h += HL) *(uint4 *)(y + h * p.yh + e) = *(const uint4 *)(x + h * p.xh + e);
            continue;
        }
        const int e = v * V;
        float c[V], s[V];
#pragma unroll
        for (int k = 0; k < V; k += N)
            rotary_angles<E, LG, N>(p, p.pos + n * p.axes, (e + k) >> LG, (e + k) & (G - 1), c + k, s + k);
#pragma unroll 2
        for (int h = h0; h < p.H; h += HL) {
            float a[V], b[V];
            EL::unpack(*(const uint4 *)(x + h * p.xh + e), a);
            EL::unpack(*(const uint4 *)(x + h * p.xh + PG + e), b);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float t = a[k] * c[k] - b[k] * s[k];
                b[k] = fmaf(a[k], s[k], b[k] * c[k]);
                a[k] = t;
            }
            *(uint4 *)(y + h * p.yh + e) = EL::pack(a);
            *(uint4 *)(y + h * p.yh + PG + e) = EL::pack(b);
        }
    }
}

// Any alignment: one lane a channel pair with all its group elements.
template <class E, int LG>
__global__ void __launch_bounds__(256) k_rotary_any(const RotaryParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    constexpr int G = 1 << LG;
    const int work = p.dc - p.P;  // pairs, then the channels that are copied
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < p.N * work; id += (int64_t)gridDim.x * 256) {
        const int64_t n = id / work;
        const int j = (int)(id - n * work);
        const T *x = (const T *)p.x + n * p.xt + j * G;
        T *y = (T *)p.y + n * p.yt + j * G;
        const int PG = p.P * G;
        float c[G], s[G];
        if (j < p.P) rotary_angles<E, LG, G>(p, p.pos + n * p.axes, j, 0, c, s);
        for (int h = 0; h < p.H; ++h) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float b = EL::get(x[h * p.xh + PG + g]);
                if (j >= p.P) {
                    y[h * p.yh + PG + g] = EL::put(b);
                } else {
                    const float a = EL::get(x[h * p.xh + g]);
                    y[h * p.yh + g] = EL::put(a * c[g] - b * s[g]);
                    y[h * p.yh + PG + g] = EL::put(fmaf(a, s[g], b * c[g]));
                }
            }
        }
    }
}

template <class E, int LG>
hipError_t run_rotary(const RotaryParams &p, hipStream_t st) {
    constexpr int V = Elem<E>::V;
    const int PG = p.P << p.lg, D = p.dc << p.lg;
    const bool copy = p.y != p.x;
    const bool vec = PG % V == 0 && D % V == 0 && p.xt % V == 0 && p.xh % V == 0 && p.yt % V == 0 && p.yh % V == 0 &&
                     (uintptr_t)p.x % 16 == 0 && (uintptr_t)p.y % 16 == 0;
    if (!vec) {
        const int64_t lanes = p.N * (p.dc - p.P);
        hipLaunchKernelGGL((k_rotary_any<E, LG>), dim3((unsigned)std::min<int64_t>((lanes + 255) / 256, 1 << 22)), dim3(256), 0, st, p);
        return hipGetLastError();
    }
    const int nv = PG / V, nr = copy ? (D - 2 * PG) / V : 0;
    // heads side by side: two waves a token, so that lanes cover whole stretches of it and an angle still serves two or
    // more heads (12544 tokens, 32 heads of 16 x 8: 38 us when chosen, against 45 us at half and 39 us at twice); all of them where
    // there are few tokens
    const int64_t few = (int64_t)device_num_cus() * 512;
    int HL = std::min(p.H, std::max(1, 128 / (nv + nr)));
    while (HL < p.H && p.N * (nv + nr) * HL < few) HL = std::min(p.H, HL * 2);
    const int64_t lanes = p.N * (nv + nr) * HL;
    hipLaunchKernelGGL((k_rotary<E, LG>), dim3((unsigned)std::min<int64_t>((lanes + 255) / 256, 1 << 22)), dim3(256), 0, st, p, nv, nr, HL);
    return hipGetLastError();
}

template <class E>
hipError_t run_rotary_e(const RotaryParams &p, hipStream_t s) {
    switch (p.lg) {
        case 0: return run_rotary<E, 0>(p, s);
        case 1: return run_rotary<E, 1>(p, s);
        case 2: return run_rotary<E, 2>(p, s);
        default: return run_rotary<E, 3>(p, s);
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryParams &p, eqlin_dtype_t dtype, hipStream_t s) {
    if (dtype == EQLIN_F32) return run_rotary_e<F32>(p, s);
    if (dtype == EQLIN_F16) return run_rotary_e<F16>(p, s);
    return run_rotary_e<BF16>(p, s);
}

}  // namespace eqlin

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
// Bound by memory: x read once, y written once, in 16-byte vectors.
#include "stage.h"

namespace eqlin {

namespace {

// cos and sin of one pair's angle for group element g
template <class E>
__device__ __forceinline__ void rotary_angle(const RotaryParams &p, const int *pos, int j, int g, float &c, float &s) {
    int axis = 0;
    while (axis + 1 < p.axes && j >= p.end[axis]) ++axis;
    double at;
    const int back = p.axes - axis;  // 2: rows, 1: columns
    if (p.axes > 1 && back <= 2 && p.lg > 0) {
        const double row = pos[p.axes - 2], col = pos[p.axes - 1];
        const int a = p.d4 ? (g & 3) * 2 : g << (3 - p.lg);  // eighths of a turn
        const double kH = 0.70710678118654752440;
        const double cs = a == 0 ? 1.0 : a == 4 ? -1.0 : (a & 3) == 2 ? 0.0 : (a == 1 || a == 7) ? kH : -kH;
        const double sn = (a & 3) == 0 ? 0.0 : a == 2 ? 1.0 : a == 6 ? -1.0 : a < 4 ? kH : -kH;
        at = back == 2 ? row * cs + col * sn : col * cs - row * sn;
        if (p.d4 && (g & 4) && back == 1) at = -at;
    } else {
        at = pos[axis];
    }
    double t = at * p.freq[j];
    t -= rint(t);
    const float f = (float)t;
    if constexpr (__is_same(E, F32)) {
        sincospif(2.0f * f, &s, &c);
    } else {
        s = __builtin_amdgcn_sinf(f);
        c = __builtin_amdgcn_cosf(f);
    }
    if (p.inverse) s = -s;
}

// Vectors: lanes run over the vectors of a head's first half, then over heads; HL heads at a time a token.
template <class E>
__global__ void __launch_bounds__(256) k_rotary(const RotaryParams p, int nv, int nr, int HL) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    constexpr int V = EL::V;
    const int lanes = (nv + nr) * HL;  // lanes a token; nr vectors past the pairs are copied
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < p.N * lanes; id += (int64_t)gridDim.x * 256) {
    const int64_t n = id / lanes;
    const int sub = (int)(id - n * lanes), h0 = sub / (nv + nr), v = sub % (nv + nr);
    const int PG = p.P << p.lg;
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
    for (int k = 0; k < V; ++k) rotary_angle<E>(p, p.pos + n * p.axes, (e + k) >> p.lg, (e + k) & ((1 << p.lg) - 1), c[k], s[k]);
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

// Any alignment: one lane a pair element.
template <class E>
__global__ void __launch_bounds__(256) k_rotary_any(const RotaryParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    const int PG = p.P << p.lg, D = p.dc << p.lg, work = D - PG;  // pairs, then what is copied
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < p.N * work; id += (int64_t)gridDim.x * 256) {
    const int64_t n = id / work;
    const int e = (int)(id - n * work);
    const T *x = (const T *)p.x + n * p.xt;
    T *y = (T *)p.y + n * p.yt;
    if (e >= PG) {
        for (int h = 0; h < p.H; ++h) y[h * p.yh + PG + e] = x[h * p.xh + PG + e];
        continue;
    }
    float c, s;
    rotary_angle<E>(p, p.pos + n * p.axes, e >> p.lg, e & ((1 << p.lg) - 1), c, s);
    for (int h = 0; h < p.H; ++h) {
        const float a = EL::get(x[h * p.xh + e]), b = EL::get(x[h * p.xh + PG + e]);
        y[h * p.yh + e] = EL::put(a * c - b * s);
        y[h * p.yh + PG + e] = EL::put(fmaf(a, s, b * c));
    }
    }
}

template <class E>
hipError_t run_rotary(const RotaryParams &p, hipStream_t st) {
    constexpr int V = Elem<E>::V;
    const int PG = p.P << p.lg, D = p.dc << p.lg;
    const bool copy = p.y != p.x;
    const bool vec = PG % V == 0 && D % V == 0 && p.xt % V == 0 && p.xh % V == 0 && p.yt % V == 0 && p.yh % V == 0 &&
                     (uintptr_t)p.x % 16 == 0 && (uintptr_t)p.y % 16 == 0;
    if (!vec) {
        const int64_t lanes = p.N * (D - PG);
        hipLaunchKernelGGL((k_rotary_any<E>), dim3((unsigned)std::min<int64_t>((lanes + 255) / 256, 1 << 22)), dim3(256), 0, st, p);
        return hipGetLastError();
    }
    const int nv = PG / V, nr = copy ? (D - 2 * PG) / V : 0;
    // heads side by side: enough that a wave's lanes cover whole stretches of a token, and all of them where
    // there are few tokens
    const int64_t few = (int64_t)device_num_cus() * 512;
    int HL = std::min(p.H, std::max(1, 64 / (nv + nr)));
    while (HL < p.H && p.N * (nv + nr) * HL < few) HL = std::min(p.H, HL * 2);
    const int64_t lanes = p.N * (nv + nr) * HL;
    hipLaunchKernelGGL((k_rotary<E>), dim3((unsigned)std::min<int64_t>((lanes + 255) / 256, 1 << 22)), dim3(256), 0, st, p, nv, nr, HL);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotaryParams &p, eqlin_dtype_t dtype, hipStream_t s) {
    if (dtype == EQLIN_F32) return run_rotary<F32>(p, s);
    if (dtype == EQLIN_F16) return run_rotary<F16>(p, s);
    return run_rotary<BF16>(p, s);
}

}  // namespace eqlin

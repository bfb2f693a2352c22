// norm.hip -- root-mean-square norm of a token's C x G values with the residual's addition, its 8-bit
// output, and its gradients.
//
//   s = x + r;  rstd = (mean over C G of s^2 + eps)^-1/2;  y = s rstd gamma[c]
//
// The mean runs over all C G values and gamma has one value a channel, so a shift of the group axis passes
// through. Everything is held in fp32; y comes from the unrounded sum, s and y are each rounded once.
//
// Bound by memory: a row is read once into registers (one wave a row up to 64 * 16 bytes * VPT, one
// workgroup above that), reduced there, and written. Longer or unaligned rows take the element loop,
// which reads the row a second time. bf16, 25088 tokens of 96 x 4 with the residual: 14.4 us (77 MB, 5.3 TB/s; a large
// copy reaches 5.1 from memory, and part of this stays in the last cache); fp16 to 8 bits, 12544 tokens of 256 x 8: 37.8 us
// (180 MB, 4.8 TB/s). The element loop: 25088 tokens of 97 x 2, 23 us (39 MB, 1.7 TB/s).
#include "norm_rows.h"

namespace eqlin {

namespace {

// scale of a row: its largest magnitude becomes 448, the largest e4m3 value; 1 for a row of zeros, and no
// smaller than the smallest normal number, so that 1 / scale is finite
__device__ __forceinline__ float e4m3_scale(float amax) {
    return amax > 0.0f ? fmaxf(amax / 448.0f, 1.17549435e-38f) : 1.0f;
}

// y / scale as division rounds it: the product with the rounded reciprocal, corrected once by its remainder (Markstein 1990).
// The last bit of the quotient decides the code of a value halfway between two, where the reciprocal alone is off as often
// as not. (An infinite scale makes the finite values 0: no remainder is taken.) 12544 tokens of 256 x 8, fp16: 33.4 us a call,
// back to back, as with the reciprocal alone, 34.9 us with the compiler's division.
struct Divisor {
    float inv, neg;
    __device__ __forceinline__ explicit Divisor(float scale) : inv(1.0f / scale), neg(scale < INFINITY ? -scale : 0.0f) {}
    __device__ __forceinline__ float quotient(float y) const {
        const float t = y * inv;
        return fmaf(fmaf(t, neg, y), inv, t);
    }
};

// gamma of the V elements from element e on (fp32; ones without gamma)
template <class E>
__device__ __forceinline__ void load_gamma(const typename Elem<E>::T *gamma, int e, int lg, float *f) {
#pragma unroll
    for (int j = 0; j < Elem<E>::V; ++j) f[j] = gamma ? Elem<E>::get(gamma[(e + j) >> lg]) : 1.0f;
}

// f[0..V) -> V e4m3 values at dst (V-byte aligned)
template <int V>
__device__ __forceinline__ void store_e4m3(const float *f, uint8_t *dst) {
    uint32_t w[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
        int t = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j], f[4 * j + 1], 0, false);
        t = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j + 2], f[4 * j + 3], t, true);
        w[j] = (uint32_t)t;
    }
    if constexpr (V == 8) *(uint2 *)dst = make_uint2(w[0], w[1]);
    else *(uint32_t *)dst = w[0];
}

// Rows in registers: WAVES waves a row, VPT vectors a lane.
template <class E, int WAVES, int VPT, bool QUANT>
__global__ void __launch_bounds__(256) k_rmsnorm(const NormParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    constexpr int V = EL::V, LANES = 64 * WAVES, RPB = 4 / WAVES;
    __shared__ float red[4];
    RowGroup<WAVES> grp = {red};
    const int L = p.C << p.lg, lane = threadIdx.x % LANES;
    const float inv_L = 1.0f / (float)L;
    float gam[VPT][V];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * LANES + lane) * V;
        if (e < L) load_gamma<E>((const T *)p.gamma, e, p.lg, gam[v]);
    }
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LANES; row < p.N; row += (int64_t)gridDim.x * RPB) {
        const T *x = (const T *)p.x + row * L, *r = p.r ? (const T *)p.r + row * L : nullptr;
        uint4 xv[VPT], rv[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * V;
            xv[v] = e < L ? *(const uint4 *)(x + e) : make_uint4(0, 0, 0, 0);
            rv[v] = r && e < L ? *(const uint4 *)(r + e) : make_uint4(0, 0, 0, 0);
        }
        float s[VPT][V], ss = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * V;
            float t[V];
            EL::unpack(xv[v], s[v]);
            EL::unpack(rv[v], t);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[v][j] += t[j];
                ss = fmaf(s[v][j], s[v][j], ss);
            }
            if (p.sum && e < L) *(uint4 *)((T *)p.sum + row * L + e) = EL::pack(s[v]);
        }
        const float rstd = rsqrtf(grp.sum(ss) * inv_L + p.eps);
        float amax = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[v][j] *= e < L ? rstd * gam[v][j] : 0.0f;
                if constexpr (QUANT) amax = fmaxf(amax, fabsf(s[v][j]));
            }
            if constexpr (!QUANT)
                if (e < L) *(uint4 *)((T *)p.y + row * L + e) = EL::pack(s[v]);
        }
        if constexpr (QUANT) {
            amax = grp.max(amax);
            const float scale = e4m3_scale(amax);
            const Divisor by(scale);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int e = (v * LANES + lane) * V;
#pragma unroll
                for (int j = 0; j < V; ++j) s[v][j] = by.quotient(s[v][j]);
                if (e < L) store_e4m3<V>(s[v], p.q + row * L + e);
            }
            if (lane == 0) p.scale[row] = scale;
        }
        if (p.rstd && lane == 0) p.rstd[row] = rstd;
    }
}

// Any row length and alignment: one workgroup a row, element by element, the row read again for the output.
template <class E, bool QUANT>
__global__ void __launch_bounds__(256) k_rmsnorm_any(const NormParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    __shared__ float red[4];
    RowGroup<4> grp = {red};
    const int L = p.C << p.lg;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        const T *x = (const T *)p.x + row * L, *r = p.r ? (const T *)p.r + row * L : nullptr;
        float ss = 0.0f;
        for (int e = threadIdx.x; e < L; e += 256) {
            const float s = EL::get(x[e]) + (r ? EL::get(r[e]) : 0.0f);
            ss = fmaf(s, s, ss);
            if (p.sum) ((T *)p.sum)[row * L + e] = EL::put(s);
        }
        const float rstd = rsqrtf(grp.sum(ss) / (float)L + p.eps);
        float scale = 1.0f;
        if constexpr (QUANT) {
            float amax = 0.0f;
            for (int e = threadIdx.x; e < L; e += 256) {
                const float s = EL::get(x[e]) + (r ? EL::get(r[e]) : 0.0f);
                amax = fmaxf(amax, fabsf(s * (p.gamma ? rstd * EL::get(((const T *)p.gamma)[e >> p.lg]) : rstd)));
            }
            amax = grp.max(amax);
            scale = e4m3_scale(amax);
        }
        for (int e = threadIdx.x; e < L; e += 256) {
            const float s = EL::get(x[e]) + (r ? EL::get(r[e]) : 0.0f);
            const float y = s * (p.gamma ? rstd * EL::get(((const T *)p.gamma)[e >> p.lg]) : rstd);
            if constexpr (QUANT)
                p.q[row * L + e] = (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(y / scale, 0.0f, 0, false) & 0xff);
            else
                ((T *)p.y)[row * L + e] = EL::put(y);
        }
        if (threadIdx.x == 0) {
            if (p.rstd) p.rstd[row] = rstd;
            if constexpr (QUANT) p.scale[row] = scale;
        }
    }
}

// ---- gradients ----
//
//   xh = s rstd;  w = dy gamma;  dx = ds + rstd (w - xh mean(w xh));  dgamma[c] = sum over tokens and g of dy xh
//
// dx is also the gradient of the residual (both enter through the sum). A lane keeps the same columns for
// every row it takes, so dgamma's sums stay in its registers; each workgroup leaves one partial row, and
// k_norm_dgamma adds those in a fixed order (no atomics: the same bits every time). bf16, 25088 tokens of 96 x 4: 15 us
// (77 MB, 5.1 TB/s) and 4 us for the partial rows.
template <class E, int WAVES, int VPT>
__global__ void __launch_bounds__(256) k_rmsnorm_bwd(const NormGradParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    constexpr int V = EL::V, LANES = 64 * WAVES, RPB = 4 / WAVES;
    extern __shared__ float part[];  // [RPB][C] where dgamma is wanted
    __shared__ float red[4];
    RowGroup<WAVES> grp = {red};
    const int L = p.C << p.lg, lane = threadIdx.x % LANES, G = 1 << p.lg;
    const float inv_L = 1.0f / (float)L;
    float gam[VPT][V], acc[VPT][V];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * LANES + lane) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) gam[v][j] = 0.0f, acc[v][j] = 0.0f;
        if (e < L) load_gamma<E>((const T *)p.gamma, e, p.lg, gam[v]);
    }
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LANES; row < p.N; row += (int64_t)gridDim.x * RPB) {
        const int64_t at = row * L;
        uint4 sv[VPT], dv[VPT], av[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * V;
            sv[v] = e < L ? *(const uint4 *)((const T *)p.s + at + e) : make_uint4(0, 0, 0, 0);
            dv[v] = e < L ? *(const uint4 *)((const T *)p.dy + at + e) : make_uint4(0, 0, 0, 0);
            av[v] = p.ds && e < L ? *(const uint4 *)((const T *)p.ds + at + e) : make_uint4(0, 0, 0, 0);
        }
        const float rstd = p.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float s[V], d[V];
            EL::unpack(sv[v], s);
            EL::unpack(dv[v], d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float dx = d[j] * s[j] * rstd;
                dot = fmaf(dx, gam[v][j], dot);
                acc[v][j] += dx;
            }
        }
        const float mean = grp.sum(dot) * inv_L;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * V;
            float s[V], d[V], a[V];
            EL::unpack(sv[v], s);
            EL::unpack(dv[v], d);
            EL::unpack(av[v], a);
#pragma unroll
            for (int j = 0; j < V; ++j) a[j] = fmaf(rstd, fmaf(d[j], gam[v][j], -s[j] * rstd * mean), a[j]);
            if (e < L) *(uint4 *)((T *)p.dx + at + e) = EL::pack(a);
        }
    }
    if (!p.dgamma) return;
    // a channel's G values: within the vector (G <= V), or over G / V neighbouring lanes
    const int sub = threadIdx.x / LANES;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = (v * LANES + lane) * V;
        if (G > V) {  // fp32, G = 8: two lanes a channel
#pragma unroll
            for (int j = 1; j < V; ++j) acc[v][0] += acc[v][j];
            acc[v][0] += __shfl_xor(acc[v][0], 1);
            if (e < L && (lane & 1) == 0) part[sub * p.C + (e >> p.lg)] = acc[v][0];
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if ((j & (G - 1)) == 0) {
                    float t = acc[v][j];
                    if (G > 1 && j + 1 < V) t += acc[v][j + 1 < V ? j + 1 : j];
                    if (G > 2)
#pragma unroll
                        for (int k = 2; k < 4; ++k) t += acc[v][j + k < V ? j + k : j];
                    if (G > 4)
#pragma unroll
                        for (int k = 4; k < 8; ++k) t += acc[v][j + k < V ? j + k : j];
                    if (e < L) part[sub * p.C + ((e + j) >> p.lg)] = t;
                }
            }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.C; c += 256) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < RPB; ++k) t += part[k * p.C + c];
        p.part[(int64_t)blockIdx.x * p.C + c] = t;
    }
}

// Any row length and alignment; a thread owns whole channels, so its partial sums in global memory are its own.
template <class E>
__global__ void __launch_bounds__(256) k_rmsnorm_bwd_any(const NormGradParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    __shared__ float red[4];
    RowGroup<4> grp = {red};
    const int L = p.C << p.lg, G = 1 << p.lg;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        const T *s = (const T *)p.s + row * L, *dy = (const T *)p.dy + row * L;
        const float rstd = p.rstd[row];
        float dot = 0.0f;
        for (int c = threadIdx.x; c < p.C; c += 256) {
            const float g = p.gamma ? EL::get(((const T *)p.gamma)[c]) : 1.0f;
            float t = 0.0f;
            for (int j = 0; j < G; ++j) t = fmaf(EL::get(dy[c * G + j]) * rstd, EL::get(s[c * G + j]), t);
            dot = fmaf(t, g, dot);
            if (p.dgamma) {
                float *a = p.part + (int64_t)blockIdx.x * p.C + c;
                *a = first ? t : *a + t;
            }
        }
        first = false;
        const float mean = grp.sum(dot) / (float)L;
        for (int e = threadIdx.x; e < L; e += 256) {
            const float g = p.gamma ? EL::get(((const T *)p.gamma)[e >> p.lg]) : 1.0f;
            const float a = p.ds ? EL::get(((const T *)p.ds)[row * L + e]) : 0.0f;
            ((T *)p.dx)[row * L + e] = EL::put(fmaf(rstd, fmaf(EL::get(dy[e]), g, -EL::get(s[e]) * rstd * mean), a));
        }
    }
}

// dgamma[c] = sum of the workgroups' partial rows: 16 channels x 64 row groups a workgroup, each thread's loads
// independent (1024 rows of 96: 17 us with 16 groups and one load after the other, 4 us so).
__global__ void __launch_bounds__(1024) k_norm_dgamma(const float *part, int rows, int C, float *dgamma) {
    __shared__ float t[64][17];
    const int j = threadIdx.x & 15, c = blockIdx.x * 16 + j, g = threadIdx.x >> 4;
    float a = 0.0f;
    if (c < C)
#pragma unroll 8
        for (int r = g; r < rows; r += 64) a += part[(int64_t)r * C + c];
    t[g][j] = a;
    __syncthreads();
    if (threadIdx.x < 64) {  // the first wave: 4 threads a channel, 16 groups each
        const int q = threadIdx.x >> 4;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += t[16 * q + k][j];
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (q == 0 && c < C) dgamma[c] = s;
    }
}

__global__ void k_zero(float *p, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

constexpr int kBwdPerCu = 4;  // workgroups of the gradient a compute unit: also bounds the partial rows

template <class E, bool QUANT>
hipError_t run_norm(const NormParams &p, hipStream_t s) {
    constexpr int V = Elem<E>::V;
    const int64_t L = (int64_t)p.C << p.lg;
    if (L % V != 0 || L > 256 * V * 8) {
        hipLaunchKernelGGL((k_rmsnorm_any<E, QUANT>), dim3(grid_for(p.N, 1, 8)), dim3(256), 0, s, p);
        return hipGetLastError();
    }
#define EQLIN_NORM(W, VPT) \
    hipLaunchKernelGGL((k_rmsnorm<E, W, VPT, QUANT>), dim3(grid_for(p.N, 4 / W, 8)), dim3(256), 0, s, p)
    const int64_t vecs = (L / V + 63) / 64;  // vectors a lane of one wave
    if (vecs <= 1) EQLIN_NORM(1, 1);
    else if (vecs <= 2) EQLIN_NORM(1, 2);
    else if (vecs <= 4) EQLIN_NORM(1, 4);
    else if (vecs <= 8) EQLIN_NORM(4, 2);
    else if (vecs <= 16) EQLIN_NORM(4, 4);
    else EQLIN_NORM(4, 8);
#undef EQLIN_NORM
    return hipGetLastError();
}

bool bwd_in_registers(int64_t L, int V, int C) { return L % V == 0 && L <= 256 * V * 8 && C <= 8192; }

template <class E>
hipError_t run_norm_bwd(const NormGradParams &p, hipStream_t s) {
    constexpr int V = Elem<E>::V;
    const int64_t L = (int64_t)p.C << p.lg;
    if (p.N == 0) {
        if (p.dgamma) hipLaunchKernelGGL(k_zero, dim3((p.C + 255) / 256), dim3(256), 0, s, p.dgamma, p.C);
        return hipGetLastError();
    }
    unsigned grid;
    if (!bwd_in_registers(L, V, p.C)) {
        grid = grid_for(p.N, 1, kBwdPerCu);
        hipLaunchKernelGGL((k_rmsnorm_bwd_any<E>), dim3(grid), dim3(256), 0, s, p);
    } else {
#define EQLIN_NORM(W, VPT)                                                                                         \
    do {                                                                                                           \
        grid = grid_for(p.N, 4 / W, kBwdPerCu);                                                                    \
        hipLaunchKernelGGL((k_rmsnorm_bwd<E, W, VPT>), dim3(grid), dim3(256), p.dgamma ? (4 / W) * p.C * 4 : 0, s, p); \
    } while (0)
        const int64_t vecs = (L / V + 63) / 64;
        if (vecs <= 1) EQLIN_NORM(1, 1);
        else if (vecs <= 2) EQLIN_NORM(1, 2);
        else if (vecs <= 4) EQLIN_NORM(1, 4);
        else if (vecs <= 8) EQLIN_NORM(4, 2);
        else if (vecs <= 16) EQLIN_NORM(4, 4);
        else EQLIN_NORM(4, 8);
#undef EQLIN_NORM
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.dgamma) return e;
    hipLaunchKernelGGL(k_norm_dgamma, dim3((p.C + 15) / 16), dim3(1024), 0, s, p.part, (int)grid, p.C, p.dgamma);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const NormParams &p, eqlin_dtype_t dtype, hipStream_t s) {
    if (p.q) {
        if (dtype == EQLIN_F32) return run_norm<F32, true>(p, s);
        if (dtype == EQLIN_F16) return run_norm<F16, true>(p, s);
        return run_norm<BF16, true>(p, s);
    }
    if (dtype == EQLIN_F32) return run_norm<F32, false>(p, s);
    if (dtype == EQLIN_F16) return run_norm<F16, false>(p, s);
    return run_norm<BF16, false>(p, s);
}

size_t rmsnorm_backward_workspace_bytes(int64_t N, int C, int) {
    return N <= 0 ? 0 : (size_t)std::min<int64_t>(N, (int64_t)device_num_cus() * kBwdPerCu) * C * sizeof(float);
}

hipError_t launch_rmsnorm_backward(const NormGradParams &p, eqlin_dtype_t dtype, hipStream_t s) {
    if (dtype == EQLIN_F32) return run_norm_bwd<F32>(p, s);
    if (dtype == EQLIN_F16) return run_norm_bwd<F16>(p, s);
    return run_norm_bwd<BF16>(p, s);
}

}  // namespace eqlin

// layernorm.hip -- layer norm of a token's C x G values with the residual's addition, and its gradients.
//
//   s = x + r;  mean = (sum of s) / (C G);  rstd = (mean over C G of (s - mean)^2 + eps)^-1/2
//   y = (s - mean) rstd gamma[c] + beta[c]
//
// Mean and variance run over all C G values, and gamma and beta have one value a channel, so a shift of the group axis
// passes through. Everything is held in fp32; the variance is taken about the mean (the row stays in registers for
// it), since E s^2 - mean^2 loses all bits of a row whose common part is large. y comes from the unrounded sum, s and
// y are each rounded once.
//
// Bound by memory: a row is read once into registers (a wave a row up to two 16-byte loads a lane, four waves to eight
// times that, sixteen above), reduced there, and written; longer rows take the element loop. Kernel times: bf16, 12544 tokens
// of 256 x 8 with the residual 36 us (205 MB, 5.7 TB/s: part of it stays in the last cache; a large copy reaches 5.0 to 5.1);
// 25088 tokens of 96 x 4 17 us (77 MB, 4.5 TB/s), their gradients 16 us and 4 us for the partial rows of gamma's and beta's;
// fp32 rows of 181, by 4-byte loads, 8.4 and 10.4 us (36 MB each way, 4.3 and 3.5 TB/s).
#include <type_traits>

#include "norm_rows.h"

namespace eqlin {

namespace {

// two sums over the lanes that share a row, in one exchange
template <int WAVES>
__device__ __forceinline__ void sum_two(float *red, float &a, float &b) {
    a = wave_sum(a), b = wave_sum(b);
    if constexpr (WAVES > 1) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a, red[WAVES + (threadIdx.x >> 6)] = b;
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) a += red[w], b += red[WAVES + w];
    }
}

// Channels of a lane's W elements, and the channel of each. LG: log2 of G where that is a constant of the kernel (16-byte
// loads: a channel's G values then share one gamma, one beta and one sum of each), else -1 (an element by itself).
template <int W, int LG>
struct Channels {
    static constexpr int N = LG < 0 ? W : (W >> LG) > 0 ? W >> LG : 1;
    static __device__ __forceinline__ constexpr int of(int j) { return LG < 0 ? j : j >> LG; }
    // the first element of channel c among the lane's
    static __device__ __forceinline__ constexpr int first(int c) { return LG < 0 ? c : c << LG; }
};

// threads of a workgroup whose rows take WAVES waves each
constexpr int threads_of(int waves) { return waves > 4 ? 64 * waves : 256; }

// Rows in registers: WAVES waves a row, VPT loads of W elements a lane.
template <class E, int W, int LG, int WAVES, int VPT>
__global__ void __launch_bounds__(threads_of(WAVES)) k_layernorm(const LayerNormParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    typedef Pack<E, W> PK;
    typedef Channels<W, LG> CH;
    constexpr int LANES = 64 * WAVES, RPB = threads_of(WAVES) / LANES;
    __shared__ float red[WAVES];
    RowGroup<WAVES> grp = {red};
    const int L = p.C << p.lg, lane = threadIdx.x % LANES;
    const float inv_L = 1.0f / (float)L;
    float gam[VPT][CH::N], bet[VPT][CH::N];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int c = 0; c < CH::N; ++c) {
            const int e = (v * LANES + lane) * W + CH::first(c);
            gam[v][c] = p.gamma && e < L ? EL::get(((const T *)p.gamma)[e >> p.lg]) : 1.0f;
            bet[v][c] = p.beta && e < L ? EL::get(((const T *)p.beta)[e >> p.lg]) : 0.0f;
        }
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LANES; row < p.N; row += (int64_t)gridDim.x * RPB) {
        const T *x = (const T *)p.x + row * L, *r = p.r ? (const T *)p.r + row * L : nullptr;
        PK xv[VPT], rv[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * W;
            xv[v].clear(), rv[v].clear();
            if (e < L) xv[v].load(x + e);
            if (r && e < L) rv[v].load(r + e);
        }
        float s[VPT][W], t = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * W;
            float add[W];
            xv[v].unpack(s[v]);
            rv[v].unpack(add);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                s[v][j] += add[j];
                t += s[v][j];
            }
            if (p.sum && e < L) PK::store((T *)p.sum + row * L + e, s[v]);
        }
        const float mean = grp.sum(t) / (float)L;  // divided: the mean of equal values is their value, a shorter sum allowing
        t = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const bool in = (v * LANES + lane) * W < L;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                s[v][j] = in ? s[v][j] - mean : 0.0f;
                t = fmaf(s[v][j], s[v][j], t);
            }
        }
        const float rstd = rsqrtf(grp.sum(t) * inv_L + p.eps);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * W;
#pragma unroll
            for (int j = 0; j < W; ++j) s[v][j] = fmaf(s[v][j] * rstd, gam[v][CH::of(j)], bet[v][CH::of(j)]);
            if (e < L) PK::store((T *)p.y + row * L + e, s[v]);
        }
        if (lane == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
    }
}

// Rows too long for the registers: one workgroup a row, element by element, x and r read three times.
template <class E>
__global__ void __launch_bounds__(256) k_layernorm_any(const LayerNormParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    __shared__ float red[4];
    RowGroup<4> grp = {red};
    const int L = p.C << p.lg;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        const T *x = (const T *)p.x + row * L, *r = p.r ? (const T *)p.r + row * L : nullptr;
        auto at = [&](int e) { return EL::get(x[e]) + (r ? EL::get(r[e]) : 0.0f); };
        float t = 0.0f;
        for (int e = threadIdx.x; e < L; e += 256) t += at(e);
        const float mean = grp.sum(t) / (float)L;
        t = 0.0f;
        for (int e = threadIdx.x; e < L; e += 256) {
            const float s = at(e), d = s - mean;
            t = fmaf(d, d, t);
            if (p.sum) ((T *)p.sum)[row * L + e] = EL::put(s);
        }
        const float rstd = rsqrtf(grp.sum(t) / (float)L + p.eps);
        for (int e = threadIdx.x; e < L; e += 256) {
            const float g = p.gamma ? EL::get(((const T *)p.gamma)[e >> p.lg]) : 1.0f;
            const float b = p.beta ? EL::get(((const T *)p.beta)[e >> p.lg]) : 0.0f;
            ((T *)p.y)[row * L + e] = EL::put(fmaf((at(e) - mean) * rstd, g, b));
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
    }
}

// ---- gradients ----
//
//   xh = (s - mean) rstd;  w = dy gamma;  dx = ds + rstd (w - mean(w) - xh mean(w xh))
//   dgamma[c] = sum over tokens and g of dy xh;  dbeta[c] = sum over tokens and g of dy
//
// dx is also the gradient of the residual. A lane keeps the same columns for every row it takes, so the parameters'
// sums stay in its registers; each workgroup leaves one partial row of 2 C sums, and k_params adds those in a fixed
// order (no atomics: the same bits every time).
template <class E, int W, int LG, int WAVES, int VPT>
__global__ void __launch_bounds__(threads_of(WAVES)) k_layernorm_bwd(const LayerNormGradParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    typedef Pack<E, W> PK;
    typedef Channels<W, LG> CH;
    constexpr int LANES = 64 * WAVES, RPB = threads_of(WAVES) / LANES;
    extern __shared__ float part[];  // [RPB][C] where the parameters' gradients are wanted
    __shared__ float red[2 * WAVES];
    const int L = p.C << p.lg, lane = threadIdx.x % LANES, G = 1 << p.lg;
    const float inv_L = 1.0f / (float)L;
    float gam[VPT][CH::N], dg[VPT][CH::N], db[VPT][CH::N];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int c = 0; c < CH::N; ++c) {
            const int e = (v * LANES + lane) * W + CH::first(c);
            gam[v][c] = p.gamma && e < L ? EL::get(((const T *)p.gamma)[e >> p.lg]) : 1.0f;
            dg[v][c] = db[v][c] = 0.0f;
        }
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LANES; row < p.N; row += (int64_t)gridDim.x * RPB) {
        const int64_t at = row * L;
        PK sv[VPT], dv[VPT], av[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * W;
            sv[v].clear(), dv[v].clear(), av[v].clear();
            if (e < L) sv[v].load((const T *)p.s + at + e);
            if (e < L) dv[v].load((const T *)p.dy + at + e);
            if (p.ds && e < L) av[v].load((const T *)p.ds + at + e);
        }
        const float mean = p.mean[row], rstd = p.rstd[row];
        float mw = 0.0f, mx = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float s[W], d[W], cg[CH::N], cb[CH::N];
            sv[v].unpack(s);
            dv[v].unpack(d);  // zeros past the row's end
#pragma unroll
            for (int c = 0; c < CH::N; ++c) cg[c] = cb[c] = 0.0f;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                cg[CH::of(j)] = fmaf(d[j], (s[j] - mean) * rstd, cg[CH::of(j)]);
                cb[CH::of(j)] += d[j];
            }
#pragma unroll
            for (int c = 0; c < CH::N; ++c) {
                mw = fmaf(cb[c], gam[v][c], mw);
                mx = fmaf(cg[c], gam[v][c], mx);
                dg[v][c] += cg[c];
                db[v][c] += cb[c];
            }
        }
        sum_two<WAVES>(red, mw, mx);
        mw *= inv_L, mx *= inv_L;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * W;
            float s[W], d[W], a[W];
            sv[v].unpack(s);
            dv[v].unpack(d);
            av[v].unpack(a);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float xh = (s[j] - mean) * rstd;
                a[j] = fmaf(rstd, fmaf(-xh, mx, fmaf(d[j], gam[v][CH::of(j)], -mw)), a[j]);
            }
            if (e < L) PK::store((T *)p.dx + at + e, a);
        }
    }
    if (!p.part) return;
    // what a lane holds of a channel, then the rest of its G values in the lanes beside it
    const int sub = threadIdx.x / LANES, held = LG < 0 ? 1 : min(G, W), pairs = LG < 0 ? min(G, W) : 1, outer = G / (held * pairs);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = (v * LANES + lane) * W;
            float t[CH::N];
#pragma unroll
            for (int c = 0; c < CH::N; ++c) t[c] = which ? db[v][c] : dg[v][c];
            if (LG < 0)
#pragma unroll
                for (int step = 1; step < W; step *= 2)
                    if (step < pairs)
#pragma unroll
                        for (int c = 0; c < CH::N; c += 2 * step) t[c] += t[c + step < CH::N ? c + step : c];
            for (int m = 1; m < outer; m *= 2) t[0] += __shfl_xor(t[0], m);
#pragma unroll
            for (int c = 0; c < CH::N; ++c)
                if (c % pairs == 0 && e < L && (lane & (outer - 1)) == 0) part[sub * p.C + ((e + CH::first(c)) >> p.lg)] = t[c];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.C; c += threads_of(WAVES)) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < RPB; ++k) t += part[k * p.C + c];
            p.part[((int64_t)blockIdx.x * 2 + which) * p.C + c] = t;
        }
    }
}

// Rows too long for the registers; a thread owns whole channels, so its partial sums in global memory are its own.
template <class E>
__global__ void __launch_bounds__(256) k_layernorm_bwd_any(const LayerNormGradParams p) {
    typedef Elem<E> EL;
    typedef typename EL::T T;
    __shared__ float red[8];
    const int L = p.C << p.lg, G = 1 << p.lg;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        const T *s = (const T *)p.s + row * L, *dy = (const T *)p.dy + row * L;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float mw = 0.0f, mx = 0.0f;
        for (int c = threadIdx.x; c < p.C; c += 256) {
            const float g = p.gamma ? EL::get(((const T *)p.gamma)[c]) : 1.0f;
            float t = 0.0f, b = 0.0f;
            for (int j = 0; j < G; ++j) {
                const float d = EL::get(dy[c * G + j]);
                t = fmaf(d, (EL::get(s[c * G + j]) - mean) * rstd, t);
                b += d;
            }
            mw = fmaf(b, g, mw);
            mx = fmaf(t, g, mx);
            if (p.part) {
                float *a = p.part + (int64_t)blockIdx.x * 2 * p.C + c;
                a[0] = first ? t : a[0] + t;
                a[p.C] = first ? b : a[p.C] + b;
            }
        }
        first = false;
        sum_two<4>(red, mw, mx);
        mw /= (float)L, mx /= (float)L;
        for (int e = threadIdx.x; e < L; e += 256) {
            const float g = p.gamma ? EL::get(((const T *)p.gamma)[e >> p.lg]) : 1.0f;
            const float a = p.ds ? EL::get(((const T *)p.ds)[row * L + e]) : 0.0f;
            const float xh = (EL::get(s[e]) - mean) * rstd;
            ((T *)p.dx)[row * L + e] = EL::put(fmaf(rstd, fmaf(-xh, mx, fmaf(EL::get(dy[e]), g, -mw)), a));
        }
    }
}

// dgamma and dbeta from the workgroups' partial rows [rows][2 C]: 8 columns x 128 row groups a workgroup, each thread's loads
// independent and, up to 1024 rows, all on their way at once. Without rows: zeros.
__global__ void __launch_bounds__(1024) k_params(const float *part, int rows, int C, float *dgamma, float *dbeta) {
    __shared__ float t[128][9];
    const int j = threadIdx.x & 7, c = blockIdx.x * 8 + j, g = threadIdx.x >> 3;
    float a = 0.0f;
    for (int at = g; at < rows; at += 1024) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = at + 128 * k < rows && c < 2 * C ? part[(int64_t)(at + 128 * k) * 2 * C + c] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) a += v[k];
    }
    t[g][j] = a;
    __syncthreads();
    if (threadIdx.x < 64) {  // the first wave: 8 threads a column, 16 groups each
        const int q = threadIdx.x >> 3;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += t[16 * q + k][j];
        s += __shfl_xor(s, 8);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (q == 0 && c < C && dgamma) dgamma[c] = s;
        if (q == 0 && c >= C && c < 2 * C && dbeta) dbeta[c - C] = s;
    }
}

constexpr int kBwdPerCu = 4;  // workgroups of the gradient a compute unit: also bounds the partial rows

// Workgroups for the rows, rows_per_wg at a time, at most per_cu a compute unit, all with the same number of turns.
unsigned even_grid(int64_t rows, int rows_per_wg, int per_cu) {
    const int64_t need = (rows + rows_per_wg - 1) / rows_per_wg, turns = (need + grid_for(rows, rows_per_wg, per_cu) - 1) / grid_for(rows, rows_per_wg, per_cu);
    return (unsigned)((need + turns - 1) / turns);
}

template <int A, int B>
struct Shape {
    static constexpr int waves = A, loads = B;
};
// The register form of a row of L elements, W a load: calls f with its Shape. False where the row is too long.
template <int W, bool WIDE, class F>
bool with_shape(int64_t L, F f) {
    const int64_t loads = (L / W + 63) / 64;  // loads a lane of one wave
    if (loads <= 1) f(Shape<1, 1>());
    else if (loads <= 2) f(Shape<1, 2>());
    // 16-byte loads: a workgroup a row from here on; of narrower ones a wave holds twice as many (12544 rows of 2048 bf16:
    // 53.7 us with a wave a row, 40.3 with four; 12543 rows of 181 fp32 with gradients: 26.8 and 33.7)
    else if (loads <= 4) f(std::conditional_t<WIDE, Shape<4, 1>, Shape<1, 4>>());
    else if (loads <= 8) f(Shape<4, 2>());
    else if (loads <= 16) f(Shape<4, 4>());
    else if (loads <= 32) f(Shape<16, 2>());
    else return false;
    return true;
}

template <class E, int W, int LG>
hipError_t run_form(const LayerNormParams &p, hipStream_t s) {
    const int64_t L = (int64_t)p.C << p.lg;
    const bool done = with_shape<W, (LG >= 0)>(L, [&](auto shape) {
        constexpr int WAVES = shape.waves, VPT = shape.loads, T = threads_of(WAVES);
        hipLaunchKernelGGL((k_layernorm<E, W, LG, WAVES, VPT>), dim3(even_grid(p.N, T / 64 / WAVES, WAVES > 4 ? 2 : 8)), dim3(T), 0, s, p);
    });
    if (!done) hipLaunchKernelGGL((k_layernorm_any<E>), dim3(grid_for(p.N, 1, 8)), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <class E, int W, int LG>
hipError_t run_form(const LayerNormGradParams &p, hipStream_t s) {
    const int64_t L = (int64_t)p.C << p.lg;
    unsigned grid = 0;
    if (p.N > 0) {
        // (the partial sums of C channels in LDS: 32 KiB at most)
        const bool done = p.C <= 8192 && with_shape<W, (LG >= 0)>(L, [&](auto shape) {
            constexpr int WAVES = shape.waves, VPT = shape.loads, T = threads_of(WAVES), RPB = T / 64 / WAVES;
            grid = even_grid(p.N, RPB, WAVES > 4 ? 1 : kBwdPerCu);
            hipLaunchKernelGGL((k_layernorm_bwd<E, W, LG, WAVES, VPT>), dim3(grid), dim3(T), p.part ? RPB * p.C * 4 : 0, s, p);
        });
        if (!done) {
            grid = grid_for(p.N, 1, kBwdPerCu);
            hipLaunchKernelGGL((k_layernorm_bwd_any<E>), dim3(grid), dim3(256), 0, s, p);
        }
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(p.dgamma || p.dbeta)) return e;
    hipLaunchKernelGGL(k_params, dim3((2 * p.C + 7) / 8), dim3(1024), 0, s, p.part, (int)grid, p.C, p.dgamma, p.dbeta);
    return hipGetLastError();
}

// Elements of a lane's load: 16 bytes where rows are whole vectors, else 4 bytes, else one.
template <class E, class P>
hipError_t run(const P &p, hipStream_t s) {
    constexpr int V = Elem<E>::V;
    const int64_t L = (int64_t)p.C << p.lg;
    if (L % V == 0) {
        switch (p.lg) {
        case 0: return run_form<E, V, 0>(p, s);
        case 1: return run_form<E, V, 1>(p, s);
        case 2: return run_form<E, V, 2>(p, s);
        default: return run_form<E, V, 3>(p, s);
        }
    }
    if constexpr (!__is_same(E, F32))
        if (L % 2 == 0) return run_form<E, 2, -1>(p, s);
    return run_form<E, 1, -1>(p, s);
}

template <class P>
hipError_t run_type(const P &p, eqlin_dtype_t dtype, hipStream_t s) {
    if (dtype == EQLIN_F32) return run<F32>(p, s);
    if (dtype == EQLIN_F16) return run<F16>(p, s);
    return run<BF16>(p, s);
}

}  // namespace

hipError_t launch_layernorm(const LayerNormParams &p, eqlin_dtype_t dtype, hipStream_t s) { return run_type(p, dtype, s); }

size_t layernorm_backward_workspace_bytes(int64_t N, int C, int) {
    return N <= 0 ? 0 : (size_t)std::min<int64_t>(N, (int64_t)device_num_cus() * kBwdPerCu) * 2 * C * sizeof(float);
}

hipError_t launch_layernorm_backward(const LayerNormGradParams &p, eqlin_dtype_t dtype, hipStream_t s) { return run_type(p, dtype, s); }

}  // namespace eqlin

// block_norm.cu -- the norms around an attention block, fused with its gate and its residual.
//
// After the block, per head row of width D (gated norm):
//     y = x r w act(g),            r = (mean(x^2) + eps)^(-1/2),   act = silu or sigmoid (or 1)
//     t = dy act(g) w:  dx = r (t - xn mean(t xn)),  dg = dy xn w act'(g),  dw = sum dy act(g) xn
// with xn = x r; before the next one, per token row of width D (residual norm):
//     x' = x + c y,   n = x' r w
//     t = dn w:  dx = dx' + r (t - xn mean(t xn)),  dy = c dx,  dw = sum dn xn,  dc = sum dx y
// The bracket cancels at an element that carries its row (D = 1: all but eps r^2 t is lost).  With ' for sums without
// the element it is also t u - xn w, u = r^2 (eps + sum' x^2 / D), w = r sum' t x / D, which does not cancel.  An element
// of more than half of the row's squares takes this form.  There is at most one, and only rows that have one form their
// two sums again, without it (taken from the sums with it they would have lost it already).  What it costs is the
// search: 2 % of the gradient of 4096 fp32 rows of 2048, 12 % at 16,384, where registers spill.
//
// All are bound by HBM: every element is read once and written once, a row lives in registers
// between its sum of squares and its output, and everything is computed in fp32 and rounded once.
// A row belongs to L lanes of a warp (2 to 32, so that narrow rows still fill 16-byte loads) or
// to a whole CTA; element e of a row is always held by the same thread, so the backward sums
// of dw and dc stay in that thread's registers over all its rows and meet once at the end: per CTA
// in shared memory, then over the CTAs by a second small kernel, in a fixed order (no atomics).
//
// Measured, bf16: gated norm of 32,768 x 32 rows of 128: 123 us, 6.6 TB/s; its gradient, 4096 x 16 rows of 128: 18 us
// (84 MB, 12.4 us at the copy rate: some 40 instructions an element are the other bound); residual norm of 256
// rows of 4096: 3.2 us; its gradient, 4096 rows of 2048, fp32 stream, learned scale: 33 us (151 MB, 22.3 us at the
// copy rate; the two launches' ends are the rest).
#include <algorithm>

#include "norm_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// V consecutive elements as they lie in memory (16-byte pieces), their values, and back.
template <typename T, int V> struct Pack {
    static constexpr int N = V * (int)sizeof(T) / 16;
    struct Raw {
        uint4 w[N];
    };
    static __device__ __forceinline__ Raw zero() {
        Raw r;
#pragma unroll
        for (int i = 0; i < N; ++i) r.w[i] = make_uint4(0, 0, 0, 0);
        return r;
    }
    static __device__ __forceinline__ Raw get(const T *p) {
        Raw r;
#pragma unroll
        for (int i = 0; i < N; ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
        return r;
    }
    static __device__ __forceinline__ void open(const Raw &r, float (&x)[V]) {
        const uint32_t *u = &r.w[0].x;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 4)
                x[i] = __uint_as_float(u[i]);
            else
                x[i] = __uint_as_float((i & 1) ? (u[i / 2] & 0xffff0000u) : (u[i / 2] << 16));
        }
    }
    static __device__ __forceinline__ void load(const T *p, float (&x)[V]) { open(get(p), x); }
    static __device__ __forceinline__ void store(T *p, const float (&x)[V]) {
        Raw r;
        uint32_t *u = &r.w[0].x;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 4) {
                u[i] = __float_as_uint(x[i]);
            } else if (!(i & 1)) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[i], x[i + 1]);
                u[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
    }
};
template <typename T> struct Pack<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ Raw zero() { return from_f32<T>(0.f); }
    static __device__ __forceinline__ Raw get(const T *p) { return *p; }
    static __device__ __forceinline__ void open(const Raw &r, float (&x)[1]) { x[0] = to_f32(r); }
    static __device__ __forceinline__ void load(const T *p, float (&x)[1]) { x[0] = to_f32(*p); }
    static __device__ __forceinline__ void store(T *p, const float (&x)[1]) { *p = from_f32<T>(x[0]); }
};

// Offset of a head row in an array of strides (t, h); contiguous arrays need no division, which would
// cost more than the row's arithmetic.
__device__ __forceinline__ long row_at(const NormView &v, long row, int H, int D, bool flat) {
    if (flat) return row * D;
    const long t = row / H;
    return t * v.t + (row - t * H) * v.h;
}

// Sum over the L threads of a row: lanes of a warp (L <= 32) or the whole CTA (L = blockDim).
// `s` holds one float per warp; consecutive calls alternate between two of them.
// `any`: whether a thread of the warp (L <= 32) or of the CTA brings it (`s` then holds twice as many floats).
template <int L>
__device__ __forceinline__ float row_sum(float x, float *s, bool *any = nullptr) {
#pragma unroll
    for (int off = (L < 32 ? L : 32) / 2; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if constexpr (L <= 32) {
        if (any) *any = __any_sync(0xffffffffu, *any);
    } else {
        if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
        if (any) {
            const bool mine = __any_sync(0xffffffffu, *any);
            if ((threadIdx.x & 31) == 0) s[L / 32 + (threadIdx.x >> 5)] = mine ? 1.f : 0.f;
        }
        __syncthreads();
        if (any) *any = __any_sync(0xffffffffu, s[L / 32 + (threadIdx.x & (L / 32 - 1))] != 0.f);
        x = s[threadIdx.x & (L / 32 - 1)];
#pragma unroll
        for (int off = L / 64; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    }
    return x;
}

// s = 1 / (1 + e), e = 2^(-a log2 e): approximate operations that flush what is below 2^-126 (a sigmoid of -88 or
// less), without the scaling that keeps subnormals, which every element would pay for.  An exponent p = a log2 e rounded
// to fp32 is off by up to 2^-24 |p|, 3e-6 of e at |a| = 80: a bf16 result does not show that; for fp32 (T) what p lost,
// which an FMA gives exactly, and what the constant lost, go in to the first order, 2^-d = 1 - d ln 2.  `rest`: 1 - s =
// e s, with all its bits where s is next to 1 (and 1 where e is infinite).
template <typename T>
__device__ __forceinline__ float sigmoid(float a, float &rest) {
    constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.925963033e-8f, kLn2 = 0.6931471805599453f;
    const float p = kLog2e * a;
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-p));
    if constexpr (sizeof(T) == 4) {
        const float low = fmaf(kLog2eLow, a, fmaf(kLog2e, a, -p));
        e = fabsf(p) < 126.f ? fmaf(e, -kLn2 * low, e) : e;     // beyond it e is 0 or infinite, or a NaN
    }
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    rest = fminf(e * s, 1.f);
    return s;
}

// act(a).  kind: 1 silu, 2 sigmoid.
template <typename T>
__device__ __forceinline__ float act_of(float a, int kind) {
    float rest;
    const float s = sigmoid<T>(a, rest);
    return kind == 1 ? a * s : s;
}

// t - xn mean(t xn) of the element that carries the row (see above), from the row's sums without it
__device__ __forceinline__ float carrier_back(float t, float x, float r, float ss1, float dot1, float eps, float inv_d) {
    return t * (r * r * fmaf(ss1, inv_d, eps)) - x * r * (r * dot1 * inv_d);
}

// ------------------------------------------------------------------------------ gated norm
// L lanes per row (256 / L rows per CTA at a time), NJ packs of V elements per lane.
// The CTAs go round the rows; a thread's next two rows are in flight, unopened, while it works on one.
template <typename T, int V, int L, int NJ>
__global__ void __launch_bounds__(kThreads) gated_norm_fwd_kernel(GatedNorm a) {
    constexpr int RPB = kThreads / L, AH = NJ == 1 ? 2 : 1;
    using Pk = Pack<T, V>;
    const int l = threadIdx.x % L;
    typename Pk::Raw x[AH][NJ], g[AH][NJ];
    float w[NJ][V];
    auto fetch = [&](int k, long row) {
        const bool live = row < a.rows;
        const T *xp = static_cast<const T *>(a.x.p) + row_at(a.x, live ? row : 0, a.H, a.D, a.flat);
        const T *gp = static_cast<const T *>(a.g.p) + row_at(a.g, live ? row : 0, a.H, a.D, a.flat);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = (l + L * j) * V;
            x[k][j] = g[k][j] = Pk::zero();
            if (live && e < a.D) {
                x[k][j] = Pk::get(xp + e);
                if (a.act) g[k][j] = Pk::get(gp + e);
            }
        }
    };
    const long step = gridDim.x * (long)RPB, first = blockIdx.x * (long)RPB + threadIdx.x / L;
#pragma unroll
    for (int k = 0; k < AH; ++k) fetch(k, first + k * step);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = (l + L * j) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) w[j][i] = 0.f;
        if (e < a.D) Pack<float, V>::load(a.w + e, w[j]);
    }
    // whole CTAs go on together (the sums use every lane of a warp)
    for (long row0 = first; row0 - threadIdx.x / L < a.rows; row0 += AH * step) {
#pragma unroll
        for (int k = 0; k < AH; ++k) {
            const long row = row0 + k * step;
            float v[NJ][V], ga[NJ][V], ss = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                Pk::open(x[k][j], v[j]);
                Pk::open(g[k][j], ga[j]);
            }
            fetch(k, row + AH * step);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(v[j][i], v[j][i], ss);
            ss = row_sum<L>(ss, nullptr);
            const float r = rsqrtf(ss * a.inv_d + a.eps);
            if (row >= a.rows) continue;
            T *yp = static_cast<T *>(a.y.p) + row_at(a.y, row, a.H, a.D, a.flat);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int e = (l + L * j) * V;
                if (e >= a.D) continue;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float y = v[j][i] * r * w[j][i];
                    if (a.act) y *= act_of<T>(ga[j][i], a.act);
                    v[j][i] = y;
                }
                Pk::store(yp + e, v[j]);
            }
        }
    }
}

// ACT, the gate's function, is a constant here: selecting it per element cost 6 %.  fp32 rows of up to 128 are held to 64
// registers, the four CTAs per SM that are launched (72 without: 37.0 us for 65,536 rows of 128 instead of 29.4).
template <typename T, int V, int L, int NJ, int ACT>
__global__ void __launch_bounds__(kThreads, V == 4 && NJ == 1 ? 4 : 1) gated_norm_bwd_kernel(GatedNorm a) {
    constexpr int RPB = kThreads / L;
    __shared__ float s_dw[RPB][L * V + 1];
    next_may_start();
    const int l = threadIdx.x % L, rg = threadIdx.x / L;
    float dw[NJ][V], w[NJ][V];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = (l + L * j) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = w[j][i] = 0.f;
        if (e < a.D) Pack<float, V>::load(a.w + e, w[j]);
    }
    using Pk = Pack<T, V>;
    typename Pk::Raw ax[NJ], ag[NJ], ad[NJ];    // the next row, in flight
    auto fetch = [&](long row) {
        const bool live = row < a.rows;
        const long rr = live ? row : 0;
        const T *xp = static_cast<const T *>(a.x.p) + row_at(a.x, rr, a.H, a.D, a.flat);
        const T *gp = static_cast<const T *>(a.g.p) + row_at(a.g, rr, a.H, a.D, a.flat);
        const T *dyp = static_cast<const T *>(a.dy.p) + row_at(a.dy, rr, a.H, a.D, a.flat);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = (l + L * j) * V;
            ax[j] = ag[j] = ad[j] = Pk::zero();
            if (live && e < a.D) {
                ax[j] = Pk::get(xp + e);
                ad[j] = Pk::get(dyp + e);
                if (ACT) ag[j] = Pk::get(gp + e);
            }
        }
    };
    fetch(blockIdx.x * (long)RPB + rg);
    for (long row0 = blockIdx.x * (long)RPB; row0 < a.rows; row0 += gridDim.x * (long)RPB) {
        const long row = row0 + rg;
        const bool live = row < a.rows;
        const long rr = live ? row : 0;
        float x[NJ][V], g[NJ][V], dy[NJ][V], ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            Pk::open(ax[j], x[j]);
            Pk::open(ag[j], g[j]);
            Pk::open(ad[j], dy[j]);
        }
        fetch(row + gridDim.x * (long)RPB);
        float sg[NJ][V], top = 0.f;             // sigmoid of the gate: its two special-function operations once
        auto t_of = [&](int j, int i) { return dy[j][i] * (ACT == 1 ? g[j][i] * sg[j][i] : sg[j][i]) * w[j][i]; };
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float rest = 0.f;
                sg[j][i] = ACT ? sigmoid<T>(g[j][i], rest) : 1.f;
                if (ACT == 2) g[j][i] = rest;   // a sigmoid's gate is not looked at again
                ss = fmaf(x[j][i], x[j][i], ss);
                dot = fmaf(t_of(j, i), x[j][i], dot);
                top = fmaxf(top, fabsf(x[j][i]));
            }
        ss = row_sum<L>(ss, nullptr);
        bool carried = top * top > 0.5f * ss;
        dot = row_sum<L>(dot, nullptr, &carried);
        const float r = rsqrtf(ss * a.inv_d + a.eps), mean = r * dot * a.inv_d;
        float carrier = 0.f;
        int at = -1;                            // the carrier's place, in the lane that holds it
        if (carried) {                          // a row of the warp has an element of more than half of its squares
            float ss1 = 0.f, dot1 = 0.f, t = 0.f, v = 0.f;
            auto take = [&](float xe, float te, int e) {
                const bool is = xe * xe > 0.5f * ss;
                ss1 += is ? 0.f : xe * xe;
                dot1 += is ? 0.f : te * xe;
                t = is ? te : t;
                v = is ? xe : v;
                at = is ? e : at;
            };
            if constexpr (NJ * V <= 16) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) take(x[j][i], t_of(j, i), (l + L * j) * V + i);
            } else {                            // wide rows have no registers to spare: read again, one by one
#pragma unroll 1
                for (int k = 0; k < NJ * V; ++k) {
                    const int e = (l + L * (k / V)) * V + k % V;
                    if (!live || e >= a.D) continue;
                    const float ge = ACT ? to_f32(static_cast<const T *>(a.g.p)[row_at(a.g, rr, a.H, a.D, a.flat) + e]) : 0.f;
                    const float act = ACT ? act_of<T>(ge, ACT) : 1.f;
                    take(to_f32(static_cast<const T *>(a.x.p)[row_at(a.x, rr, a.H, a.D, a.flat) + e]),
                         to_f32(static_cast<const T *>(a.dy.p)[row_at(a.dy, rr, a.H, a.D, a.flat) + e]) * act * a.w[e], e);
                }
            }
            ss1 = row_sum<L>(ss1, nullptr);
            dot1 = row_sum<L>(dot1, nullptr);
            carrier = r * carrier_back(t, v, r, ss1, dot1, a.eps, a.inv_d);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = (l + L * j) * V;
            if (!live || e >= a.D) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float s = sg[j][i], xn = x[j][i] * r, d = dy[j][i];
                const float ac = ACT == 1 ? g[j][i] * s : s;
                const float da = ACT == 1 ? fmaf(ac, 1.f - s, s) : s * g[j][i];
                dw[j][i] = fmaf(d * ac, xn, dw[j][i]);
                g[j][i] = d * xn * w[j][i] * da;
                x[j][i] = r * fmaf(-xn, mean, d * ac * w[j][i]);
            }
            Pack<T, V>::store(static_cast<T *>(a.dx.p) + row_at(a.dx, rr, a.H, a.D, a.flat) + e, x[j]);
            if (ACT) Pack<T, V>::store(static_cast<T *>(a.dg.p) + row_at(a.dg, rr, a.H, a.D, a.flat) + e, g[j]);
        }
        if (at >= 0)                            // over what this thread has just stored
            static_cast<T *>(a.dx.p)[row_at(a.dx, rr, a.H, a.D, a.flat) + at] = from_f32<T>(carrier);
    }
    // this CTA's share of dw, row groups in order
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) s_dw[rg][l * V + i] = dw[j][i];
        __syncthreads();
        for (int c = threadIdx.x; c < L * V; c += kThreads) {
            const int e = L * j * V + c;
            if (e >= a.D) continue;
            float sum = 0.f;
            for (int g = 0; g < RPB; ++g) sum += s_dw[g][c];
            a.part[(size_t)blockIdx.x * a.D + e] = sum;
        }
    }
}

// out[c] = sum over p of part[p, c] in a fixed order: 8 columns (a sector) x 32 strands of a CTA (32 columns to
// a CTA leave narrow rows too few of them: 3 us more with 608 partial sums of 128 columns)
__global__ void __launch_bounds__(kThreads) norm_fold_kernel(const float *part, int np, int D, float *out0, float *out1) {
    __shared__ float s[8][33];
    const int c = blockIdx.x * 8 + (threadIdx.x & 7), k = threadIdx.x >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int width = out1 ? 2 * D : D;
    wait_for_previous();
    float sum = 0.f;
    if (c < width) {
#pragma unroll 8
        for (int p = k; p < np; p += 32) sum += part[(size_t)p * width + c];
    }
    s[threadIdx.x & 7][k] = sum;
    __syncthreads();
    sum = s[warp][lane];                        // column `warp`, a strand per lane
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const int cc = blockIdx.x * 8 + warp;
    if (lane == 0 && cc < width) (cc < D ? out0 : out1)[cc < D ? cc : cc - D] = sum;
}
cudaError_t norm_fold(const float *part, int np, int D, float *out0, float *out1, cudaStream_t st) {
    return launch_after(norm_fold_kernel, ((out1 ? 2 * D : D) + 7) / 8, kThreads, 0, st, part, np, D, out0, out1);
}

// ------------------------------------------------------------------------------ residual norm
// A row per warp (L = 32, 8 rows per CTA) or per CTA (L = threads).
template <typename TR, typename T, int V, int L, int NJ>
__global__ void __launch_bounds__(L > 32 ? L : kThreads) residual_norm_fwd_kernel(ResidualNorm a) {
    constexpr int RPB = L > 32 ? 1 : kThreads / L;
    __shared__ float s_red[L > 32 ? L / 32 : 1];
    const int l = threadIdx.x % L;
    const long row = blockIdx.x * (long)RPB + threadIdx.x / L;
    const bool live = row < a.rows;
    const TR *xp = static_cast<const TR *>(a.x) + (live ? row : 0) * a.xs;
    const T *yp = static_cast<const T *>(a.y) + (live ? row : 0) * a.ys;
    float z[NJ][V], ss = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = (l + L * j) * V;
        float y[V], c[V];
#pragma unroll
        for (int i = 0; i < V; ++i) z[j][i] = y[i] = 0.f, c[i] = a.c;
        if (live && e < a.D) {
            Pack<TR, V>::load(xp + e, z[j]);
            Pack<T, V>::load(yp + e, y);
            if (a.cv) Pack<float, V>::load(a.cv + e, c);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) z[j][i] = fmaf(c[i], y[i], z[j][i]);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(z[j][i], z[j][i], ss);
    ss = row_sum<L>(ss, s_red);
    const float r = rsqrtf(ss * a.inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = (l + L * j) * V;
        if (!live || e >= a.D) continue;
        Pack<TR, V>::store(static_cast<TR *>(a.xo) + row * a.D + e, z[j]);
        float w[V];
        Pack<float, V>::load(a.w + e, w);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] *= z[j][i] * r;
        Pack<T, V>::store(static_cast<T *>(a.n) + row * a.D + e, w);
    }
}

template <typename TR, typename T, int V, int L, int NJ>
__global__ void __launch_bounds__(L > 32 ? L : kThreads) residual_norm_bwd_kernel(ResidualNorm a) {
    constexpr int RPB = L > 32 ? 1 : kThreads / L;
    constexpr int SW = L > 32 ? L / 32 : 1;
    __shared__ float s_red[2][5 * SW];
    __shared__ float s_dw[L > 32 ? 1 : RPB][L > 32 ? 1 : L * V + 1];
    next_may_start();
    const int l = threadIdx.x % L, rg = threadIdx.x / L;
    float dw[NJ][V], dc[NJ][V];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = dc[j][i] = 0.f;
    // the next row's loads go out before this row is summed, where the registers hold two rows
    constexpr bool kAhead = NJ * V <= 16 && L <= 256;
    struct Row {
        typename Pack<TR, V>::Raw x[NJ], dx[NJ];
        typename Pack<T, V>::Raw dn[NJ], y[NJ];
    };
    // Fetched ahead in packs the loads have no branches, past the end the last places are read again: they go out together
    // and none is waited for early (4096 rows of 2048 fp32: 32.6 us, with branches 39.6)
    constexpr bool kClamp = kAhead && V > 1;
    auto fetch = [&](Row &r, long row) {
        const bool live = row < a.rows;
        const long rr = live ? row : kClamp ? a.rows - 1 : 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e0 = (l + L * j) * V, e = kClamp ? min(e0, a.D - V) : e0;
            r.x[j] = r.dx[j] = Pack<TR, V>::zero();
            r.dn[j] = r.y[j] = Pack<T, V>::zero();
            if (kClamp || (live && e < a.D)) {
                r.x[j] = Pack<TR, V>::get(static_cast<const TR *>(a.x) + rr * a.xs + e);
                r.dn[j] = Pack<T, V>::get(static_cast<const T *>(a.dn) + rr * a.dns + e);
                if (a.dxo) r.dx[j] = Pack<TR, V>::get(static_cast<const TR *>(a.dxo) + rr * a.dxs + e);
                if (a.y) r.y[j] = Pack<T, V>::get(static_cast<const T *>(a.y) + rr * a.ys + e);
            }
        }
    };
    Row ahead;
    if constexpr (kAhead) fetch(ahead, blockIdx.x * (long)RPB + rg);
    int turn = 0;   // the sums of consecutive rows use two sets of shared floats
    for (long row0 = blockIdx.x * (long)RPB; row0 < a.rows; row0 += gridDim.x * (long)RPB, turn ^= 1) {
        const long row = row0 + rg;
        const bool live = row < a.rows;
        float ss = 0.f, dot = 0.f, top = 0.f;
        Row r0;
        if constexpr (kAhead) {
            r0 = ahead;
            fetch(ahead, row + gridDim.x * (long)RPB);
        } else {
            fetch(r0, row);
        }
        float x[NJ][V], dn[NJ][V], dx[NJ][V], y[NJ][V];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            Pack<TR, V>::open(r0.x[j], x[j]);
            Pack<T, V>::open(r0.dn[j], dn[j]);
            Pack<TR, V>::open(r0.dx[j], dx[j]);
            Pack<T, V>::open(r0.y[j], y[j]);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = (l + L * j) * V;
            if (e >= a.D) continue;
            float w[V];
            Pack<float, V>::load(a.w + e, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ss = fmaf(x[j][i], x[j][i], ss);
                dot = fmaf(dn[j][i] * w[i], x[j][i], dot);
                top = fmaxf(top, fabsf(x[j][i]));
            }
        }
        ss = row_sum<L>(ss, s_red[turn]);
        bool carried = top * top > 0.5f * ss;
        dot = row_sum<L>(dot, s_red[turn] + SW, &carried);
        const float r = rsqrtf(ss * a.inv_d + a.eps), mean = r * dot * a.inv_d;
        float carrier = 0.f;
        int at = -1;                            // the carrier's place among this thread's elements
        if (carried) {                          // an element has more than half of its row's squares
            float ss1 = 0.f, dot1 = 0.f, t = 0.f, v = 0.f;
            auto take = [&](float xe, float te, int k) {
                const bool is = xe * xe > 0.5f * ss;
                ss1 += is ? 0.f : xe * xe;
                dot1 += is ? 0.f : te * xe;
                t = is ? te : t;
                v = is ? xe : v;
                at = is ? k : at;
            };
            if constexpr (kAhead) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int e = (l + L * j) * V;
                    if (e >= a.D) continue;
                    float w[V];
                    Pack<float, V>::load(a.w + e, w);
#pragma unroll
                    for (int i = 0; i < V; ++i) take(x[j][i], dn[j][i] * w[i], j * V + i);
                }
            } else {                            // wide rows have no registers to spare: read again, one by one
#pragma unroll 1
                for (int k = 0; k < NJ * V; ++k) {
                    const int e = (l + L * (k / V)) * V + k % V;
                    if (live && e < a.D)
                        take(to_f32(static_cast<const TR *>(a.x)[row * a.xs + e]),
                             to_f32(static_cast<const T *>(a.dn)[row * a.dns + e]) * a.w[e], k);
                }
            }
            ss1 = row_sum<L>(ss1, s_red[turn] + 3 * SW);
            dot1 = row_sum<L>(dot1, s_red[turn] + 4 * SW);
            carrier = carrier_back(t, v, r, ss1, dot1, a.eps, a.inv_d);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = (l + L * j) * V;
            if (!live || e >= a.D) continue;
            float w[V], c[V];
            Pack<float, V>::load(a.w + e, w);
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = a.c;
            if (a.cv) Pack<float, V>::load(a.cv + e, c);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xn = x[j][i] * r;
                dw[j][i] = fmaf(dn[j][i], xn, dw[j][i]);
                float b = fmaf(-xn, mean, dn[j][i] * w[i]);
                b = at == j * V + i ? carrier : b;
                dx[j][i] += r * b;
                dc[j][i] = fmaf(dx[j][i], y[j][i], dc[j][i]);
                c[i] *= dx[j][i];
            }
            Pack<TR, V>::store(static_cast<TR *>(a.xo) + row * a.D + e, dx[j]);
            Pack<T, V>::store(static_cast<T *>(a.n) + row * a.D + e, c);
        }
    }
    const int width = a.y ? 2 * a.D : a.D;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which == 1 && !a.y) break;
        float *part = a.part + (size_t)blockIdx.x * width + which * a.D;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            if constexpr (L > 32) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = (l + L * j) * V + i;
                    if (e < a.D) part[e] = which ? dc[j][i] : dw[j][i];
                }
            } else {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < V; ++i) s_dw[rg][l * V + i] = which ? dc[j][i] : dw[j][i];
                __syncthreads();
                for (int c = threadIdx.x; c < L * V; c += kThreads) {
                    const int e = L * j * V + c;
                    if (e >= a.D) continue;
                    float sum = 0.f;
                    for (int g = 0; g < RPB; ++g) sum += s_dw[g][c];
                    part[e] = sum;
                }
            }
        }
    }
}

template <typename T, int V, int L, int NJ>
cudaError_t gated_go(const GatedNorm &a, bool bwd, cudaStream_t st) {
    const long blocks = (a.rows + kThreads / L - 1) / (kThreads / L);
    if (!bwd) {
        if (blocks > 0x7fffffffL) return cudaErrorInvalidValue;
        gated_norm_fwd_kernel<T, V, L, NJ><<<(unsigned)std::min(blocks, 8L * a.sms), kThreads, 0, st>>>(a);
        return cudaGetLastError();
    }
    // what its registers let an SM hold (8, in two rounds, cost 8 % more with 65,536 rows of 128)
    const int grid = (int)std::min(blocks, 4L * a.sms);
    if (a.act == 0)
        gated_norm_bwd_kernel<T, V, L, NJ, 0><<<grid, kThreads, 0, st>>>(a);
    else if (a.act == 1)
        gated_norm_bwd_kernel<T, V, L, NJ, 1><<<grid, kThreads, 0, st>>>(a);
    else
        gated_norm_bwd_kernel<T, V, L, NJ, 2><<<grid, kThreads, 0, st>>>(a);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    return norm_fold(a.part, grid, a.D, a.dw, nullptr, st);
}

// The narrowest lane group whose 16-byte packs cover the row; whole warps with several packs
// above that; single elements where a size or an address does not allow 16 bytes.
template <typename T>
cudaError_t gated_pick(const GatedNorm &a, bool vec, bool bwd, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    if (vec) {
        const int packs = a.D / V;
        if (packs <= 4) return gated_go<T, V, 4, 1>(a, bwd, st);
        if (packs <= 8) return gated_go<T, V, 8, 1>(a, bwd, st);
        if (packs <= 16) return gated_go<T, V, 16, 1>(a, bwd, st);
        if (packs <= 32) return gated_go<T, V, 32, 1>(a, bwd, st);
        if (packs <= 64) return gated_go<T, V, 32, 2>(a, bwd, st);
        if constexpr (V == 4)   // fp32 rows of more than 512
            if (packs > 128) return gated_go<T, V, 32, 8>(a, bwd, st);
        return gated_go<T, V, 32, 4>(a, bwd, st);
    }
    if (a.D <= 128) return gated_go<T, 1, 32, 4>(a, bwd, st);
    if (a.D <= 256) return gated_go<T, 1, 32, 8>(a, bwd, st);
    return gated_go<T, 1, 32, 32>(a, bwd, st);
}

template <typename TR, typename T, int V, int L, int NJ>
cudaError_t residual_go(const ResidualNorm &a, bool bwd, cudaStream_t st) {
    constexpr int threads = L > 32 ? L : kThreads, rpb = threads / L;
    const long blocks = (a.rows + rpb - 1) / rpb;
    if (!bwd) {
        if (blocks > 0x7fffffffL) return cudaErrorInvalidValue;
        residual_norm_fwd_kernel<TR, T, V, L, NJ><<<(unsigned)blocks, threads, 0, st>>>(a);
        return cudaGetLastError();
    }
    // a partial sum of dw (and dc) per CTA costs as much traffic as rows do: two CTAs of a row per SM, which the
    // prefetched row keeps busy; narrow rows (a warp each) have narrow partial sums
    const int grid = (int)std::min(blocks, (long)(L > 32 ? 2 : 8) * a.sms);
    residual_norm_bwd_kernel<TR, T, V, L, NJ><<<grid, threads, 0, st>>>(a);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    return norm_fold(a.part, grid, a.D, a.dw, a.y ? a.dc : nullptr, st);
}

template <typename TR, typename T>
cudaError_t residual_pick(const ResidualNorm &a, bool vec, bool bwd, cudaStream_t st) {
    if (vec) {
        const int packs = a.D / 8;
        if (packs <= 32) return residual_go<TR, T, 8, 32, 1>(a, bwd, st);
        if (packs <= 64) return residual_go<TR, T, 8, 32, 2>(a, bwd, st);
        if (packs <= 256) return residual_go<TR, T, 8, 256, 1>(a, bwd, st);
        if (packs <= 512) return residual_go<TR, T, 8, 256, 2>(a, bwd, st);
        if (packs <= 1024) return residual_go<TR, T, 8, 512, 2>(a, bwd, st);
        return residual_go<TR, T, 8, 512, 4>(a, bwd, st);
    }
    if (a.D <= 256) return residual_go<TR, T, 1, 32, 8>(a, bwd, st);
    if (a.D <= 2048) return residual_go<TR, T, 1, 256, 8>(a, bwd, st);
    if (a.D <= 8192) return residual_go<TR, T, 1, 512, 16>(a, bwd, st);
    return residual_go<TR, T, 1, 512, 32>(a, bwd, st);
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNorm &a0, bool bwd, cudaStream_t st) {
    const int V = a0.dtype == DType::BF16 ? 8 : 4;
    GatedNorm a = a0;
    bool vec = a.D % V == 0;
    a.flat = 1;
    for (const NormView *v : {&a.x, &a.g, &a.y, &a.dy, &a.dx, &a.dg})
        if (v->p && (v->t != (long long)a.H * a.D || (a.H > 1 && v->h != a.D))) a.flat = 0;
    for (const NormView *v : {&a.x, &a.g, &a.y, &a.dy, &a.dx, &a.dg})
        if (v->p && ((reinterpret_cast<uintptr_t>(v->p) & 15) || v->t % V || v->h % V)) vec = false;
    if (reinterpret_cast<uintptr_t>(a.w) & 15) vec = false;
    return a.dtype == DType::BF16 ? gated_pick<__nv_bfloat16>(a, vec, bwd, st) : gated_pick<float>(a, vec, bwd, st);
}

cudaError_t launch_residual_norm(const ResidualNorm &a, bool bwd, cudaStream_t st) {
    bool vec = a.D % 8 == 0 && a.xs % 8 == 0 && a.ys % 8 == 0 && a.dns % 8 == 0 && a.dxs % 8 == 0;
    for (const void *p : {a.x, a.y, a.dn, a.dxo, (const void *)a.xo, (const void *)a.n, (const void *)a.w, (const void *)a.cv})
        if (reinterpret_cast<uintptr_t>(p) & 15) vec = false;
    if (a.res == DType::F32 && a.dtype == DType::BF16) return residual_pick<float, __nv_bfloat16>(a, vec, bwd, st);
    if (a.dtype == DType::BF16) return residual_pick<__nv_bfloat16, __nv_bfloat16>(a, vec, bwd, st);
    return residual_pick<float, float>(a, vec, bwd, st);
}

}  // namespace kda

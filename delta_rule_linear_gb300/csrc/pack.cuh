// pack.cuh -- 16-byte packs of elements and the sigmoid, shared by the kernels that go over rows of channels.
#pragma once

#include "kda_internal.cuh"

namespace kda {

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

}  // namespace kda

// ssm_math.cuh -- the scalar functions of the state space scan.
#pragma once

#include "pack.cuh"

namespace kda {

constexpr float kLog2eF = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// softplus(z) = max(z, 0) + log1p(e), e = exp(-|z|) in [0, 1].  A time step of 1e-3 needs log1p's relative accuracy, which
// the logarithm of 1 + e has lost: log1p(e) / e is a polynomial of degree 9 (fitted to its values on [0, 1] with the
// largest relative error least, 5e-9; evaluated in fp32 1.6e-7).  The product |z| log2 e is rounded to fp32, 2^-24 |p|
// ln 2 of e: a bf16 z does not carry that, for fp32 (T) it goes in to the first order.
template <typename T>
__device__ __forceinline__ float softplus(float z) {
    constexpr float kLow = 1.925963033e-8f, kLn2 = 0.6931471805599453f;
    const float m = fabsf(z), p = kLog2eF * m;
    float e = ex2(-p);
    if constexpr (sizeof(T) == 4) {
        const float low = fmaf(kLow, m, fmaf(kLog2eF, m, -p));
        e = p < 126.f ? fmaf(e, -kLn2 * low, e) : e;
    }
    float q = -0.0032440253999084234f;
    q = fmaf(q, e, 0.01985146477818489f);
    q = fmaf(q, e, -0.056959543377161026f);
    q = fmaf(q, e, 0.10603656619787216f);
    q = fmaf(q, e, -0.15305593609809875f);
    q = fmaf(q, e, 0.1967594027519226f);
    q = fmaf(q, e, -0.24954134225845337f);
    q = fmaf(q, e, 0.3332996368408203f);
    q = fmaf(q, e, -0.4999990165233612f);
    q = fmaf(q, e, 1.f);
    return fmaf(q, e, fmaxf(z, 0.f)) + (z != z ? z : 0.f);     // fmaxf drops a NaN
}

}  // namespace kda

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

// Two fp32 in one register pair: the packed operations do both in one instruction.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void each(Two x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// softplus(z) = max(z, 0) + log1p(e), e = exp(-|z|) in [0, 1], of two.  A time step of 1e-3 needs log1p's relative accuracy,
// which the logarithm of 1 + e has lost: log1p(e) / e is a polynomial of degree 9 (fitted to its values on [0, 1] with the
// largest relative error least, 5e-9; evaluated in fp32 1.6e-7).  The product |z| log2 e is rounded to fp32, 2^-24 |p|
// ln 2 of e: a bf16 z does not carry that, for fp32 (T) it goes in to the first order.  A NaN comes through e.
template <typename T>
__device__ __forceinline__ float softplus_e(float z) {
    constexpr float kLow = 1.925963033e-8f, kLn2 = 0.6931471805599453f;
    const float m = fabsf(z), p = kLog2eF * m;
    float e = ex2(-p);
    if constexpr (sizeof(T) == 4) {
        const float low = fmaf(kLow, m, fmaf(kLog2eF, m, -p));
        e = p < 126.f ? fmaf(e, -kLn2 * low, e) : e;
    }
    return e;
}
template <typename T>
__device__ __forceinline__ void softplus(float &z0, float &z1) {
    constexpr float c[10] = {-0.0032440253999084234f, 0.01985146477818489f, -0.056959543377161026f, 0.10603656619787216f, -0.15305593609809875f, 0.1967594027519226f, -0.24954134225845337f, 0.3332996368408203f, -0.4999990165233612f, 1.f};
    const Two e = two(softplus_e<T>(z0), softplus_e<T>(z1));
    Two q = two(c[0], c[0]);
#pragma unroll
    for (int i = 1; i < 10; ++i) q = fma2(q, e, two(c[i], c[i]));
    each(fma2(q, e, two(fmaxf(z0, 0.f), fmaxf(z1, 0.f))), z0, z1);
}
template <typename T>
__device__ __forceinline__ float softplus(float z) {
    float other = 0.f;
    softplus<T>(z, other);
    return z;
}

// N consecutive elements as words, unopened: one load where VEC (aligned to the smaller of 16 bytes and all of them), the
// first `n` of them one by one otherwise.
template <typename T, int N> struct Few {
    static constexpr int W = N * (int)sizeof(T) / 4 ? N * (int)sizeof(T) / 4 : 1;
    uint32_t w[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void set(int i, T x) {
        if constexpr (sizeof(T) == 4)
            w[i] = __float_as_uint(x);
        else
            w[i / 2] |= (uint32_t)__bfloat16_as_ushort(x) << 16 * (i & 1);
    }
    template <bool VEC> __device__ __forceinline__ void load(const T *p, int n) {
        zero();
        if (VEC) {
            if (n <= 0) return;
            if constexpr (W % 4 == 0) {
#pragma unroll
                for (int i = 0; i < W / 4; ++i) {
                    const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
                    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
                }
            } else if constexpr (W == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                w[0] = v.x, w[1] = v.y;
            } else if constexpr (N * sizeof(T) == 4) {
                w[0] = *reinterpret_cast<const uint32_t *>(p);
            } else {
                set(0, p[0]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < n) set(i, p[i]);
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else
            return __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    }
    // as they are, to an aligned place
    __device__ __forceinline__ void keep(T *p) const {
        if constexpr (N == 1) {
            if constexpr (sizeof(T) == 4)
                p[0] = __uint_as_float(w[0]);
            else
                p[0] = __ushort_as_bfloat16((unsigned short)w[0]);
        } else if constexpr (W % 4 == 0) {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (W == 2) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        }
    }
    template <bool VEC> static __device__ __forceinline__ void store(T *p, const float (&x)[N], int n) {
        if (VEC) {
            if (n <= 0) return;
            Few r;
            r.zero();
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < N; ++i) r.w[i] = __float_as_uint(x[i]);
            } else if constexpr (N > 1) {
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[i], x[i + 1]);
                    r.w[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
            if constexpr (N == 1)
                p[0] = from_f32<T>(x[0]);
            else if constexpr (W % 4 == 0)
#pragma unroll
                for (int i = 0; i < W / 4; ++i)
                    reinterpret_cast<uint4 *>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
            else if constexpr (W == 2)
                *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
            else
                *reinterpret_cast<uint32_t *>(p) = r.w[0];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < n) p[i] = from_f32<T>(x[i]);
        }
    }
};

__device__ __forceinline__ uint32_t shared_at(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// BYTES from global to shared memory behind the thread's back, zeros behind the first `have` of them.
template <int BYTES> __device__ __forceinline__ void copy_async(void *to, const void *from, int have) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(shared_at(to)), "l"(from), "r"(have) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(shared_at(to)), "l"(from), "n"(BYTES), "r"(have) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

// N elements of each of THREADS threads in shared memory, copied there and read again by the thread itself (no barrier):
// 16-byte units of the threads side by side.
template <typename T, int N, int THREADS> struct Own {
    static constexpr int BYTES = N * (int)sizeof(T), UNIT = BYTES < 16 ? BYTES : 16, UNITS = BYTES / UNIT;
    static constexpr int SIZE = BYTES * THREADS;
    static constexpr int PER = UNIT / (int)sizeof(T);       // elements of a unit
    // VEC: p is aligned to a unit and n is 0 or N; otherwise the first n elements, by twos where `pairs` (p aligned to two).
    // What is not there is not touched.
    template <bool VEC> static __device__ __forceinline__ void fetch(uint8_t *slot, int tid, const T *p, int n, bool pairs) {
        uint8_t *to = slot + tid * UNIT;
        if constexpr (VEC) {
#pragma unroll
            for (int u = 0; u < UNITS; ++u) copy_async<UNIT>(to + u * UNIT * THREADS, p + u * PER, n > 0 ? UNIT : 0);
        } else if (sizeof(T) == 4 || pairs) {
            constexpr int E = 4 / (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < N; i += E)
                copy_async<4>(to + i / PER * UNIT * THREADS + i % PER * (int)sizeof(T), p + i,
                              i >= n ? 0 : i + E <= n ? 4 : 4 / E);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                *reinterpret_cast<T *>(to + i / PER * UNIT * THREADS + i % PER * (int)sizeof(T)) = i < n ? p[i] : from_f32<T>(0.f);
        }
    }
    static __device__ __forceinline__ Few<T, N> read(const uint8_t *slot, int tid) {
        Few<T, N> r;
        const uint8_t *at = slot + tid * UNIT;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const uint8_t *q = at + u * UNIT * THREADS;
            if constexpr (UNIT == 16) {
                const uint4 v = *reinterpret_cast<const uint4 *>(q);
                r.w[4 * u] = v.x, r.w[4 * u + 1] = v.y, r.w[4 * u + 2] = v.z, r.w[4 * u + 3] = v.w;
            } else if constexpr (UNIT == 8) {
                const uint2 v = *reinterpret_cast<const uint2 *>(q);
                r.w[0] = v.x, r.w[1] = v.y;
            } else {
                r.w[0] = *reinterpret_cast<const uint32_t *>(q);
            }
        }
        return r;
    }
};

}  // namespace kda
